// keyweights.cuh: the attention weight that each key of a prompt received,
//   w[b,hk,j] = sum over the G query heads of hk, sum over queries i of the counted rows whose
//               band holds j, of exp(scale q_i . k_j - lse_i),
// from the log-sum-exp that the training forward writes. The rows counted are the last
// `last` of the stream's n tokens: max(0, n - last) <= i < n. Keys at or past n get 0.
//
// key_weights_tc_kernel (bf16): tcgen05 score tiles, below.
// key_weights_simt_kernel (fp32): FMA on 64-key x 64-query score tiles. A CTA, or a cluster that
// splits the query tiles, owns 64 keys, so every sum has one owner and a fixed order. Small
// calls are bound by the latency of a tile's loads (2 streams, 4 heads, 777 tokens, D 80, W 200:
// 24 us; 2 heads of 2000 tokens, W 2000: 54 us with clusters of 8, 213 without), large ones by
// instruction issue (16 heads of 2000 tokens, D 64, W 1000, 3 GFLOP of multiply-adds: 160 us).
#pragma once
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "cache.cuh"
#include "decode.cuh"
#include "prefill_pp.cuh"
#include "ptx.cuh"
#include "umma.h"

namespace swa {

constexpr int kKwTile = 64;   // keys and queries of a score tile
constexpr int kKwDepth = 32;  // head columns staged at a time
constexpr int kKwSimtThreads = 128;

__global__ void __launch_bounds__(kKwSimtThreads, 3)
    key_weights_simt_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ lse,
                            const int64_t* __restrict__ lens, float* __restrict__ out, int64_t qsb, int64_t qsh,
                            int64_t qst, int64_t ksb, int64_t ksh, int64_t kst, int H, int Hkv, int T, int D, int W,
                            int last, float scale, int n_kt, int C, int* status) {
    constexpr int kLoads = kKwTile * kKwDepth / kKwSimtThreads;  // of q, and of k, a thread and chunk
    constexpr int kStep = kKwSimtThreads / 32;  // rows between a thread's loads
    __shared__ __align__(16) float sq[2][kKwDepth][kKwTile + 4], sk[2][kKwDepth][kKwTile + 4];  // by turns
    __shared__ __align__(16) float sl[2][kKwTile], sm_sum[kKwTile];
    const int tid = threadIdx.x, rank = (int)(blockIdx.x % C);
    const int64_t unit = blockIdx.x / C, bh = unit / n_kt;
    const int64_t b = bh / Hkv, hk = bh - b * Hkv;
    const int j0 = (int)(unit % n_kt) * kKwTile;
    const int G = H / Hkv;
    const int n = stream_len(lens, b, T, status);
    const int tq = tid & 15, tk = tid >> 4;  // this thread: queries 4 tq .., keys 8 tk ..
    // queries that see a key of the tile, cut to the counted rows; T and W are at most 2^29
    const int i_lo = max(j0, n - last), i_hi = min(n - 1, j0 + kKwTile - 1 + W - 1);
    const int per_head = j0 < n && i_hi >= i_lo ? (i_hi - i_lo + kKwTile) / kKwTile : 0;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // Query tiles rank, rank + C, .. of the G * per_head (head gh of the group, tile at of it);
    // each in chunks of kKwDepth head columns, the next chunk's loads in flight during this one's
    // products.
    int gh = 0, at = rank;
    auto settle = [&] {
        while (gh < G && at >= per_head) {
            at -= per_head;
            ++gh;
        }
    };
    if (per_head == 0) gh = G;
    settle();
    float rq[kLoads], rk[kLoads], rl = 0.f;
    const int r0 = tid >> 5, lane = tid & 31;
    const float* kb = k + b * ksb + hk * ksh + (int64_t)(j0 + r0) * kst + lane;
    auto fetch = [&](int d0) {
        const int64_t h = hk * G + gh;
        const int i0 = i_lo + kKwTile * at;
        const float* qp = q + b * qsb + h * qsh + (int64_t)(i0 + r0) * qst + d0 + lane;
        const float* kp = kb + d0;
        const bool in = d0 + lane < D;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            rq[x] = in && i0 + r0 + kStep * x <= i_hi ? *qp : 0.f;
            rk[x] = in && j0 + r0 + kStep * x < n ? *kp : 0.f;
            qp += kStep * qst;
            kp += kStep * kst;
        }
        if (d0 == 0 && tid < kKwTile) rl = i0 + tid <= i_hi ? lse[(b * H + h) * T + i0 + tid] : 0.f;
    };
    int chunk = 0, tile = 0;  // buffers
    if (gh < G) fetch(0);
    while (gh < G) {
        const int i0 = i_lo + kKwTile * at;
        float c[8][4] = {};
        const int ltile = tile;
        for (int d0 = 0; d0 < D; d0 += kKwDepth, chunk ^= 1) {
            // The buffer was last read two chunks ago, before the barrier of the chunk between.
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                sq[chunk][lane][r0 + kStep * x] = rq[x];
                sk[chunk][lane][r0 + kStep * x] = rk[x];
            }
            if (d0 == 0 && tid < kKwTile) sl[tile][tid] = rl;
            __syncthreads();
            if (d0 + kKwDepth < D) {
                fetch(d0 + kKwDepth);
            } else {
                at += C;
                tile ^= 1;
                settle();
                if (gh < G) fetch(0);
            }
            const int dn = min(kKwDepth, D - d0);  // in steps of 8: the columns past D hold zeros
            for (int d8 = 0; d8 < dn; d8 += 8) {
#pragma unroll
                for (int d = d8; d < d8 + 8; ++d) {
                    const float4 x = *reinterpret_cast<const float4*>(&sq[chunk][d][4 * tq]);
                    const float4 y = *reinterpret_cast<const float4*>(&sk[chunk][d][8 * tk]);
                    const float4 z = *reinterpret_cast<const float4*>(&sk[chunk][d][8 * tk + 4]);
                    const float xs[4] = {x.x, x.y, x.z, x.w}, ys[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int f = 0; f < 4; ++f) c[e][f] = fmaf(ys[e], xs[f], c[e][f]);
                }
            }
        }
        const float4 l4 = *reinterpret_cast<const float4*>(&sl[ltile][4 * tq]);
        const float ls[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int i = i0 + 4 * tq + f, j = j0 + 8 * tk + e;
                if (i <= i_hi && i >= j && i - j < W) sum[e] += expf(fmaf(c[e][f], scale, -ls[f]));
            }
    }
    // the 16 lanes that share a key are neighbours in one half of a warp
#pragma unroll
    for (int x = 8; x > 0; x >>= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], x);
    if (tq == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sm_sum[8 * tk + e] = sum[e];
    }
    if (C > 1) {
        ptx::cluster_arrive();
        ptx::cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank == 0 && tid < kKwTile && j0 + tid < T) {
        float x[8];  // all loads in flight together
#pragma unroll
        for (int r = 0; r < 8; ++r) x[r] = r < C ? ptx::cluster_ld(ptx::cluster_addr(sm_sum + tid, r)) : 0.f;
        float w = C > 1 ? x[0] : sm_sum[tid];
#pragma unroll
        for (int r = 1; r < 8; ++r) w += x[r];
        out[bh * T + j0 + tid] = w;
    }
    if (C > 1) {  // the other CTAs' sums are read before they leave
        ptx::cluster_arrive();
        ptx::cluster_wait();
    }
}

// ------------------------------------------------------------------ bf16, tensor cores
// key_weights_tc_kernel: a CTA owns 128 keys, the rows of S^T = K Q^T, so that a thread's TMEM
// lane is a key and its sum needs no exchange: no maximum, no second product, no atomics. The
// queries that see the tile's keys come in slices of 64 rows (a head of the group, rows i0 ..),
// two to a stage of 128 columns. Stage j uses ring slot, TMEM buffer and warpgroup j & 1. A CTA
// may go on from one key tile to the next without a pause (C = 1). Roles:
//   warp 0        TMA of the key tile and the query slices (lane 0); -lse log2(e) of each stage's
//                 columns into shared memory
//   warp 1        TMEM allocation and MMA issue
//   warps 2 .. 9  two warpgroups: p = 2^(s c + nlse) and the row sums of every second stage
// Bound: one exp a band pair on the special-function unit (16 a clock and SM), 2 x the time of
// the product at D = 128. 32 heads of 16384 tokens, W 4096 (1.88 G exponentials): 0.58 to 0.62 ms
// by the clock that the power cap leaves: the unit is 0.70 busy, the issue slots 0.39, and
// what is missing is warps with scores to work on (a buffer goes back to the product when all of its
// 128 columns are read). With 1, 2, 3 or 4 of each 8 exponentials as a polynomial on the FMA pipe an
// earlier form took 588, 614, 665 and 681 us against 582. Two CTAs share an SM, so that one's
// start and end overlap the other's work. Few keys and many queries: a cluster of C CTAs splits
// the slices of one key tile and adds its sums in rank order through distributed shared memory.
constexpr int kKwThreads = 320;
constexpr int kKwSlice = 64;  // query rows of a slice
constexpr int kKwStats = 8;   // stages of nlse in shared memory
constexpr int kKwSets = 4;    // units' sums in shared memory

template <int D>
struct KwCfg {
    static_assert(D == 64 || D == 128, "head dim 64 or 128");
    static constexpr int kBoxBytes = 128 * 128;  // 128 rows x 64 bf16
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kSliceBytes = kTileBytes / 2;
    static constexpr int kRingOff = kTileBytes;
    static constexpr int kNlOff = kRingOff + 2 * kTileBytes;
    static constexpr int kRedOff = kNlOff + kKwStats * 128 * 4;  // [kKwSets][128] sums of a warpgroup
    static constexpr int kBarOff = kRedOff + kKwSets * 128 * 4;
    // k_full, ring_full[2], s_full[2], s_read[2], red_full[kKwSets][4], drain
    static constexpr int kNumBars = 8 + 4 * kKwSets;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
    static constexpr uint32_t kTmemCols = 256;
};

// What a CTA works on: the unit-th pair of key tile and (b, hk), units in ascending order of key
// tiles, so that the light ones at the end come last.
struct KwItem {
    int64_t b, hk;
    int j0, n, i_lo, i_hi;  // keys j0 .., queries i_lo .. i_hi
    int per_head;           // slices of one head
    int s0, slices, stages; // this CTA's slices of the G * per_head: s0 .. s0 + slices - 1
    __device__ __forceinline__ KwItem(int64_t unit, const int64_t* lens, int64_t BHk, int H, int Hkv, int T, int W, int last,
                                      int rank, int C, int* status) {
        const int64_t bh = unit % BHk;
        b = bh / Hkv;
        hk = bh - b * Hkv;
        j0 = (int)(unit / BHk) * 128;
        n = stream_len(lens, b, T, status);
        i_lo = max(j0, n - last);
        i_hi = min(n - 1, j0 + 127 + W - 1);  // T and W are at most 2^29
        const int rows = j0 < n ? i_hi - i_lo + 1 : 0;
        per_head = rows > 0 ? (rows + kKwSlice - 1) / kKwSlice : 0;
        const int64_t all = (int64_t)per_head * (H / Hkv);
        s0 = (int)(all * rank / C);
        slices = (int)(all * (rank + 1) / C) - s0;
        stages = (slices + 1) / 2;
    }
};

// The r-th unit of CTA (or cluster) g of G, in a snake order that evens out slowly changing work.
__device__ __forceinline__ int64_t kw_unit(int64_t r, int64_t g, int64_t G) { return r * G + ((r & 1) ? G - 1 - g : g); }

// Sums of 16 columns of a row: v scores, nl the columns' nlse; EDGE: only those whose bit of
// mask is set count.
template <bool EDGE>
__device__ __forceinline__ void kw_sum16(const uint32_t (&v)[16], const float* nl, float c2, uint32_t mask,
                                         ptx::f32x2 (&acc)[2]) {
    const ptx::f32x2 cc = {c2, c2};
#pragma unroll
    for (int t = 0; t < 16; t += 4) {
        const float4 n4 = *reinterpret_cast<const float4*>(nl + t);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int x = t + 2 * u;
            const ptx::f32x2 z = ptx::fma2({__uint_as_float(v[x]), __uint_as_float(v[x + 1])}, cc,
                                           u ? ptx::f32x2{n4.z, n4.w} : ptx::f32x2{n4.x, n4.y});
            ptx::f32x2 p = {ptx::ex2(z.x), ptx::ex2(z.y)};
            if (EDGE) p = {mask & (1u << x) ? p.x : 0.f, mask & (2u << x) ? p.y : 0.f};
            acc[u] = ptx::add2(acc[u], p);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kKwThreads, 2)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const float* __restrict__ lse, const int64_t* __restrict__ lens, float* __restrict__ out,
                          int64_t units, int H, int Hkv, int T, int W, int last, float c2, int C, uint64_t wait_limit_ns, int* status) {
    using Cf = KwCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Cf::kBarOff);
    uint64_t* ring_full = k_full + 1;   // [2]
    uint64_t* s_full = ring_full + 2;   // [2] the scores of a stage (and so its ring slot is free), and its nlse
    uint64_t* s_read = s_full + 2;      // [2] the scores of a buffer are in registers
    uint64_t* red_full = s_read + 2;    // [kKwSets][4] a unit's sums of one warpgroup, by TMEM quarter
    uint64_t* drain = red_full + 4 * kKwSets;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cf::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cf::kMiscOff + 4);
    float* sm_nl = reinterpret_cast<float*>(smem + Cf::kNlOff);
    float* sm_red = reinterpret_cast<float*>(smem + Cf::kRedOff);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int rank = (int)(blockIdx.x % C);
    const int64_t BHk = units / ((T + 127) / 128), step = gridDim.x / C;

    if (tid == 0) {
        ptx::mbar_init(k_full, 1);
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(ring_full + x, 1);
            ptx::mbar_init(s_full + x, 2);
            ptx::mbar_init(s_read + x, 4);
        }
        for (int x = 0; x < 4 * kKwSets; ++x) ptx::mbar_init(red_full + x, 1);
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, Cf::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint32_t J = 0;         // stages of the units before, in every role
    uint32_t n_k = 0;       // units with a stage so far
    bool ok = true;

    if (warp == 0) {
        // -------------------------------------------------------------------- loads, nlse
        for (int64_t r = 0, u; ok && (u = kw_unit(r, blockIdx.x / C, step)) < units; ++r) {
            const KwItem it(u, lens, BHk, H, Hkv, T, W, last, rank, C, status);
            if (it.stages == 0) continue;
            // The slices in order: of the loads (at, head) and, two stages ahead, of the lse (lat,
            // row), which are read long before they are stored.
            int at = it.s0 % it.per_head, head = (int)it.hk * (H / Hkv) + it.s0 / it.per_head;
            int lat = at, left = it.slices;
            const float* row = lse + ((int64_t)it.b * H + head) * T + lane;
            float a[2][4];
            auto fetch = [&](float (&v)[4]) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    v[2 * x] = v[2 * x + 1] = INFINITY;
                    if (left > 0) {
                        const int i = it.i_lo + kKwSlice * lat;
                        if (i + lane <= it.i_hi) v[2 * x] = row[i];
                        if (i + 32 + lane <= it.i_hi) v[2 * x + 1] = row[i + 32];
                        --left;
                        if (++lat == it.per_head) {
                            lat = 0;
                            row += T;
                        }
                    }
                }
            };
            fetch(a[0]);
            fetch(a[1]);
            for (int jj = 0; jj < it.stages && ok; jj += 2) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int j = jj + z;
                    if (j >= it.stages || !ok) break;
                    const uint32_t y = J & 1;
                    // Stage J - 2 has its scores: ring slot y is free, and so is the nlse slot of stage
                    // J - 8: those scores were computed after the warpgroup had read stage J - 4's,
                    // which it does after it has finished stage J - 6. Before the first stage of a
                    // unit stage J - 1 has too, so that the key tile may be replaced.
                    const uint32_t P = j == 0 ? J - 1 : J - 2;
                    if (J >= (j == 0 ? 1u : 2u))
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full + (P & 1), (P >> 1) & 1, wait_limit_ns, abort_flag));
                    if (!ok) break;
                    if (lane == 0) {
                        if (j == 0) {
                            ptx::mbar_arrive_expect_tx(k_full, Cf::kTileBytes);
                            for (int c = 0; c < D / 64; ++c)
                                ptx::tma_load_4d(smem + c * Cf::kBoxBytes, &tm_k, k_full, 64 * c, it.j0, (int)it.hk, (int)it.b);
                        }
                        uint8_t* dst = smem + Cf::kRingOff + y * Cf::kTileBytes;
                        const int here = min(2, it.slices - 2 * j);
                        ptx::mbar_arrive_expect_tx(ring_full + y, here * Cf::kSliceBytes);
                        for (int x = 0; x < here; ++x) {
                            for (int c = 0; c < D / 64; ++c)
                                ptx::tma_load_4d(dst + c * Cf::kBoxBytes + x * (Cf::kBoxBytes / 2), &tm_q, ring_full + y,
                                                 64 * c, it.i_lo + kKwSlice * at, head, (int)it.b);
                            if (++at == it.per_head) {
                                at = 0;
                                ++head;
                            }
                        }
                    }
                    if (j == 0) ++n_k;
                    float* nl = sm_nl + 128 * (J % kKwStats) + lane;
#pragma unroll
                    for (int x = 0; x < 4; ++x) nl[32 * x] = a[z][x] * -1.4426950408889634f;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(s_full + y);
                    fetch(a[z]);
                    ++J;
                }
            }
        }
        if (!ok && lane == 0) {
            atomicCAS(status, 0, 5);
            *abort_flag = 1;
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------------- MMA issuer
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, wait_limit_ns, abort_flag));
        };
        const uint64_t desc_hi = umma::smem_desc(0, 0, 1024) & 0xFFFFFFFF00000000ull;
        const uint32_t lo = (uint32_t)umma::smem_desc(0, 16, 1024);
        const uint32_t k_lo = (ptx::smem_u32(smem) >> 4) | lo;
        for (int64_t r = 0, u; ok && (u = kw_unit(r, blockIdx.x / C, step)) < units; ++r) {
            const KwItem it(u, lens, BHk, H, Hkv, T, W, last, rank, C, status);
            if (it.stages == 0) continue;
            ok = wait(k_full, n_k & 1);
            ++n_k;
            for (int j = 0; j < it.stages && ok; ++j, ++J) {
                const uint32_t y = J & 1;
                if (J >= 2) ok = wait(s_read + y, ((J >> 1) - 1) & 1);
                if (ok) ok = wait(ring_full + y, (J >> 1) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t q_lo = ((ptx::smem_u32(smem + Cf::kRingOff) + y * Cf::kTileBytes) >> 4) | lo;
                const uint32_t idesc = umma::idesc_bf16_f32(128, it.slices - 2 * j >= 2 ? 128 : 64, 0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * Cf::kBoxBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_ss_one(tmem + 128 * y, desc_hi | (k_lo + off), desc_hi | (q_lo + off), idesc,
                                    kk > 0 ? 1u : 0u);
                }
                ptx::tc_commit_one(s_full + y);
            }
        }
        if (!ok && lane == 0) {
            atomicCAS(status, 0, 5);
            *abort_flag = 1;
        }
    } else {
        // -------------------------------------------------------------------- exponentials, sums
        const int quarter = warp & 3, y = (warp - 2) >> 2, row = 32 * quarter + lane;
        const uint32_t col = tmem + ((uint32_t)(32 * quarter) << 16) + 128 * y;
        for (int64_t r = 0, u; ok && (u = kw_unit(r, blockIdx.x / C, step)) < units; ++r) {
            int jk, i_lo, per_head, slices, stages, at, full_lo, full_hi, see, n;
            const int first = (y - J) & 1;  // this warpgroup's first stage of the unit
            {
                const KwItem it(u, lens, BHk, H, Hkv, T, W, last, rank, C, status);
                jk = it.j0 + row;
                n = it.n;
                i_lo = it.i_lo;
                per_head = it.per_head;
                slices = it.slices;
                stages = it.stages;
                // a slice is full when every key of the tile is in the band of each of its rows
                full_lo = it.j0 + 127;
                full_hi = min(it.j0 + W - 1, it.i_hi) - (kKwSlice - 1);
                see = min(jk + W - 1, it.i_hi);  // this key is seen by queries jk .. see
                at = stages ? (it.s0 + 2 * first) % per_head : 0;  // slice of its head, at the stage's first
            }
            auto put = [&](float w) {  // a key past the stream's end may have met anything in its row
                if (jk < T) out[u % BHk * T + jk] = jk < n ? w : 0.f;
            };
            if (stages == 0) {
                if (C == 1) {
                    if (y == 0) put(0.f);
                } else {
                    sm_red[128 * y + row] = 0.f;
                }
                continue;
            }
            float mine = 0.f;  // by way of each stage's own sum: fewer additions to the large one
            for (int j = first; j < stages; j += 2) {
                const uint32_t Jj = J + j;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full + y, (Jj >> 1) & 1, wait_limit_ns, abort_flag));
                if (!ok) break;
                ptx::tc_fence_after();
                ptx::f32x2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
                const int at1 = at + 1 < per_head ? at + 1 : 0;
                const int i0 = i_lo + kKwSlice * at, i1 = i_lo + kKwSlice * at1;
                const bool two = slices - 2 * j >= 2;
                const bool full0 = i0 >= full_lo && i0 <= full_hi, full1 = i1 >= full_lo && i1 <= full_hi;
                const float* nl = sm_nl + 128 * (Jj % kKwStats);
                if (full0 && full1 && two) {
                    // 16 columns at a time, the next ones on their way during the arithmetic
                    uint32_t v[2][16];
                    ptx::tmem_ld16(col, v[0]);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        ptx::tmem_ld_wait();
                        ptx::reg_fence(v[x & 1]);
                        if (x < 7) {
                            ptx::tmem_ld16(col + 16 * (x + 1), v[(x + 1) & 1]);
                        } else {
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(s_read + y);
                        }
                        kw_sum16<false>(v[x & 1], nl + 16 * x, c2, 0, acc);
                    }
                } else {
                    // only the 16 columns that one of the warp's keys is seen by
#pragma unroll 1
                    for (int x = 0; x < (two ? 8 : 4); ++x) {
                        const int c0 = (x < 4 ? i0 : i1) + 16 * (x & 3);  // the query of the first column
                        const int lo = min(max(jk - c0, 0), 16), hi = min(max(see - c0 + 1, lo), 16);
                        if (!__any_sync(0xffffffffu, hi > lo)) continue;
                        uint32_t v[16];
                        ptx::tmem_ld16(col + 16 * x, v);
                        ptx::tmem_ld_wait();
                        ptx::reg_fence(v);
                        kw_sum16<true>(v, nl + 16 * x, c2, (1u << hi) - (1u << lo), acc);
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(s_read + y);
                }
                mine += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                at += 4;
                while (at >= per_head) at -= per_head;
            }
            if (!ok) break;
            if (C > 1) {
                sm_red[128 * y + row] = mine;
            } else {
                // The warpgroup that does not have the unit's last stage leaves its sums and goes
                // on; the other adds its own. There are four sets by turns: that warpgroup cannot
                // be four units ahead, for in each it either waits for the other one or leaves it
                // two stages or more, and stage J + 2 has scores only after the other's warps have
                // read stage J's.
                const uint32_t set = n_k % kKwSets;
                float* red = sm_red + 128 * set + row;
                uint64_t* full = red_full + 4 * set + quarter;
                if (((J + stages - 1) & 1) != (uint32_t)y) {
                    *red = mine;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(full);
                } else {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(full, (n_k / kKwSets) & 1, wait_limit_ns, abort_flag));
                    if (ok) put(*red + mine);
                }
            }
            J += stages;
            ++n_k;
        }
        if (!ok) {
            atomicCAS(status, 0, 5);
            *abort_flag = 1;
        }
    }

    // ------------------------------------------------------------------------ teardown
    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        if (warp == 0 && lane == 0) {
            if (n_k > 0) ptx::mbar_wait(k_full, (n_k - 1) & 1, kPPDrainLimitNs, nullptr);
            for (uint32_t y = 0; y < 2 && y < J; ++y)
                ptx::mbar_wait(ring_full + y, ((J - 1 - y) / 2) & 1, kPPDrainLimitNs, nullptr);
        }
        if (warp == 1) {
            ptx::tc_commit_one(drain);
            ptx::mbar_wait(drain, 0, kPPDrainLimitNs, nullptr);
        }
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, Cf::kTmemCols);
    }

    if (C > 1) {  // one unit a cluster: its CTAs' sums, in rank order
        ptx::cluster_arrive();
        ptx::cluster_wait();
        if (rank == 0 && tid < 128) {
            const KwItem it(blockIdx.x / C, lens, BHk, H, Hkv, T, W, last, rank, C, status);
            float x[8][2];  // all loads in flight together
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const uint32_t from = ptx::cluster_addr(sm_red + tid, r < C ? r : 0);
                x[r][0] = r < C ? ptx::cluster_ld(from) : 0.f;
                x[r][1] = r < C ? ptx::cluster_ld(from + 512) : 0.f;
            }
            float w = x[0][0] + x[0][1];
#pragma unroll
            for (int r = 1; r < 8; ++r) w += x[r][0] + x[r][1];
            const int j = it.j0 + tid;
            if (j < T) out[(it.b * Hkv + it.hk) * T + j] = j < it.n ? w : 0.f;
        }
        ptx::cluster_arrive();  // the other CTAs' sums are read before they leave
        ptx::cluster_wait();
    }
}

}  // namespace swa
