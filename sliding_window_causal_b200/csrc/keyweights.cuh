// keyweights.cuh: the attention weight that each key of a prompt received,
//   w[b,hk,j] = sum over the G query heads of hk, sum over queries i of the counted rows whose
//               band holds j, of exp(scale q_i . k_j - lse_i),
// from the log-sum-exp that the training forward writes. The rows counted are the last
// `last` of the stream's n tokens: max(0, n - last) <= i < n. Keys at or past n get 0.
//
// key_weights_tc_kernel (bf16): tcgen05 score tiles, below.
// key_weights_simt_kernel (fp32): FMA on 64-key x 64-query score tiles. One CTA owns 64 keys and runs over the query tiles and heads that see them, so every sum has one
// owner and a fixed order.
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

__global__ void __launch_bounds__(256)
    key_weights_simt_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ lse,
                            const int64_t* __restrict__ lens, float* __restrict__ out, int64_t qsb, int64_t qsh,
                            int64_t qst, int64_t ksb, int64_t ksh, int64_t kst, int H, int Hkv, int T, int D, int W,
                            int last, float scale, int n_kt, int* status) {
    __shared__ float sq[kKwDepth][kKwTile + 4], sk[kKwDepth][kKwTile + 4];
    __shared__ float sl[kKwTile];
    const int tid = threadIdx.x;
    const int64_t bh = blockIdx.x / n_kt;
    const int64_t b = bh / Hkv, hk = bh - b * Hkv;
    const int j0 = (int)(blockIdx.x % n_kt) * kKwTile;
    const int G = H / Hkv;
    const int n = stream_len(lens, b, T, status);
    const int first = n - last > 0 ? n - last : 0;
    const int tq = tid & 15, tk = tid >> 4;  // this thread: queries 4 tq .., keys 4 tk ..
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // queries that see a key of the tile: [j0, j0 + 63 + W - 1], cut to the counted rows
    const int i_lo = max(j0, first);
    const int i_hi = (int)min((int64_t)n - 1, (int64_t)j0 + kKwTile - 1 + W - 1);
    if (j0 < n) {
        for (int gh = 0; gh < G; ++gh) {
            const int64_t h = hk * G + gh;
            const float* qb = q + b * qsb + h * qsh;
            const float* kb = k + b * ksb + hk * ksh;
            for (int i0 = i_lo; i0 <= i_hi; i0 += kKwTile) {
                float c[4][4] = {};
                for (int d0 = 0; d0 < D; d0 += kKwDepth) {
                    __syncthreads();
                    for (int x = tid; x < kKwTile * kKwDepth; x += 256) {
                        const int r = x / kKwDepth, d = x % kKwDepth;
                        const bool in = d0 + d < D;
                        sq[d][r] = in && i0 + r <= i_hi ? qb[(int64_t)(i0 + r) * qst + d0 + d] : 0.f;
                        sk[d][r] = in && j0 + r < n ? kb[(int64_t)(j0 + r) * kst + d0 + d] : 0.f;
                    }
                    if (d0 == 0 && tid < kKwTile) sl[tid] = i0 + tid <= i_hi ? lse[(b * H + h) * T + i0 + tid] : 0.f;
                    __syncthreads();
#pragma unroll 8
                    for (int d = 0; d < kKwDepth; ++d) {
                        const float4 x = *reinterpret_cast<const float4*>(&sq[d][4 * tq]);
                        const float4 y = *reinterpret_cast<const float4*>(&sk[d][4 * tk]);
                        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int f = 0; f < 4; ++f) c[e][f] = fmaf(ys[e], xs[f], c[e][f]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const int i = i0 + 4 * tq + f, j = j0 + 4 * tk + e;
                        if (i <= i_hi && i >= j && i - j < W) sum[e] += expf(fmaf(c[e][f], scale, -sl[4 * tq + f]));
                    }
            }
        }
    }
    // the 16 lanes that share a key are neighbours in one half of a warp
#pragma unroll
    for (int x = 8; x > 0; x >>= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], x);
    if (tq == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j0 + 4 * tk + e < T) out[bh * T + j0 + 4 * tk + e] = sum[e];
    }
}


// ------------------------------------------------------------------ bf16, tensor cores
// key_weights_tc_kernel: a CTA owns 128 keys, the rows of S^T = K Q^T, so that a thread's TMEM
// lane is a key and its sum needs no exchange: no maximum, no second product, no atomics. The
// queries that see the tile's keys come in slices of 64 rows (a head of the group, rows i0 ..),
// two to a stage of 128 columns. Stage j uses ring slot, TMEM buffer and warpgroup j & 1. Roles:
//   warp 0        TMA of the key tile and the query slices (lane 0); -lse log2(e) of each stage's
//                 columns into shared memory
//   warp 1        TMEM allocation and MMA issue
//   warps 2 .. 9  two warpgroups: p = 2^(s c + nlse) and the row sums of every second stage
// Bound: one exp a band pair on the special-function unit (16 a clock and SM), 2 x the time of
// the product at D = 128. 32 heads of 16384 tokens, W 4096 (1.88 G exponentials): 582 us, 0.72
// of that unit's rate; with 1, 2, 3 or 4 of each 8 exponentials as a polynomial on the FMA pipe
// 588, 614, 665 and 681 us, as the warps' issue slots run out first. Two CTAs share an SM, so
// that one's start and end overlap the other's work. Few keys and many queries: a cluster of C
// CTAs splits the slices of one key tile and adds its sums in rank order through distributed
// shared memory.
constexpr int kKwThreads = 320;
constexpr int kKwSlice = 64;  // query rows of a slice
constexpr int kKwStats = 8;   // stages of nlse in shared memory

template <int D>
struct KwCfg {
    static_assert(D == 64 || D == 128, "head dim 64 or 128");
    static constexpr int kBoxBytes = 128 * 128;  // 128 rows x 64 bf16
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kSliceBytes = kTileBytes / 2;
    static constexpr int kRingOff = kTileBytes;
    static constexpr int kNlOff = kRingOff + 2 * kTileBytes;
    static constexpr int kRedOff = kNlOff + kKwStats * 128 * 4;  // [2][128] sums of the two warpgroups
    static constexpr int kBarOff = kRedOff + 2 * 128 * 4;
    static constexpr int kNumBars = 8;  // k_full, ring_full[2], s_full[2], s_read[2], drain
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
    static constexpr uint32_t kTmemCols = 256;
};

// What a CTA works on.
struct KwItem {
    int64_t b, hk;
    int j0, n, i_lo, i_hi;  // keys j0 .., queries i_lo .. i_hi
    int per_head;           // slices of one head
    int s0, s1;             // this CTA's slices of the G * per_head
    __device__ __forceinline__ int head(int s) const { return s / per_head; }
    __device__ __forceinline__ int row(int s) const { return i_lo + kKwSlice * (s % per_head); }
};

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
                          int H, int Hkv, int T, int W, int last, float c2, int C, uint64_t wait_limit_ns, int* status) {
    using Cf = KwCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Cf::kBarOff);
    uint64_t* ring_full = k_full + 1;   // [2]
    uint64_t* s_full = ring_full + 2;   // [2] the scores of a stage (and so its ring slot is free), and its nlse
    uint64_t* s_read = s_full + 2;      // [2] the scores of a buffer are in registers
    uint64_t* drain = s_read + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cf::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cf::kMiscOff + 4);
    float* sm_nl = reinterpret_cast<float*>(smem + Cf::kNlOff);
    float* sm_red = reinterpret_cast<float*>(smem + Cf::kRedOff);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    KwItem it;
    const int rank = (int)(blockIdx.x % C);
    {
        const int64_t unit = blockIdx.x / C, BHk = (int64_t)(gridDim.x / C) / ((T + 127) / 128);
        const int64_t bh = unit % BHk;  // key tiles in ascending order: the light ones at the end come last
        it.b = bh / Hkv;
        it.hk = bh - it.b * Hkv;
        it.j0 = (int)(unit / BHk) * 128;
        it.n = stream_len(lens, it.b, T, status);
        it.i_lo = max(it.j0, it.n - last);
        it.i_hi = min(it.n - 1, it.j0 + 127 + W - 1);  // T and W are at most 2^29
        const int rows = it.j0 < it.n ? it.i_hi - it.i_lo + 1 : 0;
        it.per_head = rows > 0 ? (rows + kKwSlice - 1) / kKwSlice : 0;
        const int64_t all = (int64_t)it.per_head * (H / Hkv);
        it.s0 = (int)(all * rank / C);
        it.s1 = (int)(all * (rank + 1) / C);
    }
    const int slices = it.s1 - it.s0, stages = (slices + 1) / 2;
    float sum = 0.f;  // element-wise threads: the sum of this thread's row over its stages

    if (slices > 0) {  // uniform in the CTA
        if (tid == 0) {
            ptx::mbar_init(k_full, 1);
            for (int x = 0; x < 2; ++x) {
                ptx::mbar_init(ring_full + x, 1);
                ptx::mbar_init(s_full + x, 2);
                ptx::mbar_init(s_read + x, 4);
            }
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
        uint32_t loads = 0;  // warp 0: stages whose loads are issued

        if (warp == 0) {
            // ---------------------------------------------------------------- loads, nlse
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(k_full, Cf::kTileBytes);
                for (int c = 0; c < D / 64; ++c)
                    ptx::tma_load_4d(smem + c * Cf::kBoxBytes, &tm_k, k_full, 64 * c, it.j0, (int)it.hk, (int)it.b);
            }
            bool ok = true;
            // the lse of a stage are read two stages before they are stored
            float a[2][4];
            auto fetch = [&](int j, float (&r)[4]) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int s = it.s0 + 2 * j + x;
                    r[2 * x] = r[2 * x + 1] = INFINITY;
                    if (s < it.s1) {
                        const int i = it.row(s) + lane;
                        const float* p = lse + ((int64_t)it.b * H + it.hk * (H / Hkv) + it.head(s)) * T + i;
                        if (i <= it.i_hi) r[2 * x] = p[0];
                        if (i + 32 <= it.i_hi) r[2 * x + 1] = p[32];
                    }
                }
            };
            fetch(0, a[0]);
            fetch(1, a[1]);
            for (int j0 = 0; j0 < stages && ok; j0 += 2) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = j0 + y;
                    if (j >= stages || !ok) break;
                    // Stage j - 2 has its scores: ring slot y is free, and so is the nlse slot of
                    // stage j - 8: those scores were computed after the warpgroup had read stage
                    // j - 4's, which it does after it has finished stage j - 6.
                    if (j >= 2)
                        ok = __all_sync(0xffffffffu,
                                        ptx::mbar_wait(s_full + y, ((j >> 1) - 1) & 1, wait_limit_ns, abort_flag));
                    if (!ok) break;
                    if (lane == 0) {
                        uint8_t* dst = smem + Cf::kRingOff + y * Cf::kTileBytes;
                        const int here = min(2, slices - 2 * j);
                        ptx::mbar_arrive_expect_tx(ring_full + y, here * Cf::kSliceBytes);
                        for (int x = 0; x < here; ++x) {
                            const int s = it.s0 + 2 * j + x;
                            for (int c = 0; c < D / 64; ++c)
                                ptx::tma_load_4d(dst + c * Cf::kBoxBytes + x * (Cf::kBoxBytes / 2), &tm_q, ring_full + y,
                                                 64 * c, it.row(s), (int)it.hk * (H / Hkv) + it.head(s), (int)it.b);
                        }
                    }
                    ++loads;
                    float* nl = sm_nl + 128 * (j % kKwStats) + lane;
#pragma unroll
                    for (int x = 0; x < 4; ++x) nl[32 * x] = a[y][x] * -1.4426950408889634f;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(s_full + y);
                    fetch(j + 2, a[y]);
                }
            }
            if (!ok && lane == 0) {
                atomicCAS(status, 0, 5);
                *abort_flag = 1;
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issuer
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, wait_limit_ns, abort_flag));
            };
            const uint64_t desc_hi = umma::smem_desc(0, 0, 1024) & 0xFFFFFFFF00000000ull;
            const uint32_t lo = (uint32_t)umma::smem_desc(0, 16, 1024);
            const uint32_t k_lo = (ptx::smem_u32(smem) >> 4) | lo;
            bool ok = wait(k_full, 0);
            for (int j = 0; j < stages && ok; ++j) {
                const uint32_t y = j & 1;
                if (j >= 2) ok = wait(s_read + y, ((j >> 1) - 1) & 1);
                if (ok) ok = wait(ring_full + y, (j >> 1) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t q_lo = ((ptx::smem_u32(smem + Cf::kRingOff) + y * Cf::kTileBytes) >> 4) | lo;
                const uint32_t idesc = umma::idesc_bf16_f32(128, slices - 2 * j >= 2 ? 128 : 64, 0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * Cf::kBoxBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_ss_one(tmem + 128 * y, desc_hi | (k_lo + off), desc_hi | (q_lo + off), idesc,
                                    kk > 0 ? 1u : 0u);
                }
                ptx::tc_commit_one(s_full + y);
            }
            if (!ok && lane == 0) {
                atomicCAS(status, 0, 5);
                *abort_flag = 1;
            }
        } else {
            // ---------------------------------------------------------------- exponentials, sums
            const int quarter = warp & 3, y = (warp - 2) >> 2;
            const int jk = it.j0 + 32 * quarter + lane;
            const uint32_t col = tmem + ((uint32_t)(32 * quarter) << 16) + 128 * y;
            // a slice is full when every key of the tile is in the band of each of its rows
            const int full_lo = it.j0 + 127, full_hi = min(it.j0 + W - 1, it.i_hi) - (kKwSlice - 1);
            const int see = min(jk + W - 1, it.i_hi);  // this key is seen by queries jk .. see
            int at = (it.s0 + 2 * y) % it.per_head;  // slice of its head, at the stage's first
            ptx::f32x2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
            bool ok = true;
            for (int j = y; j < stages; j += 2) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full + y, (j >> 1) & 1, wait_limit_ns, abort_flag));
                if (!ok) break;
                ptx::tc_fence_after();
                const int at1 = at + 1 < it.per_head ? at + 1 : 0;
                const int i0 = it.i_lo + kKwSlice * at, i1 = it.i_lo + kKwSlice * at1;
                const bool two = slices - 2 * j >= 2;
                const bool full0 = i0 >= full_lo && i0 <= full_hi, full1 = i1 >= full_lo && i1 <= full_hi;
                const float* nl = sm_nl + 128 * (j % kKwStats);
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
#pragma unroll 1
                    for (int x = 0; x < (two ? 8 : 4); ++x) {
                        uint32_t v[16];
                        ptx::tmem_ld16(col + 16 * x, v);
                        ptx::tmem_ld_wait();
                        ptx::reg_fence(v);
                        const int c0 = (x < 4 ? i0 : i1) + 16 * (x & 3);  // the query of the first column
                        const int lo = min(max(jk - c0, 0), 16), hi = min(max(see - c0 + 1, lo), 16);
                        kw_sum16<true>(v, nl + 16 * x, c2, (1u << hi) - (1u << lo), acc);
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(s_read + y);
                }
                at += 4;
                while (at >= it.per_head) at -= it.per_head;
            }
            sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
            if (!ok) {
                atomicCAS(status, 0, 5);
                *abort_flag = 1;
            }
        }

        // -------------------------------------------------------------------- teardown
        ptx::tc_fence_before();
        __syncthreads();
        if (*abort_flag) {
            if (warp == 0 && lane == 0) {
                ptx::mbar_wait(k_full, 0, kPPDrainLimitNs, nullptr);
                for (uint32_t y = 0; y < 2 && y < loads; ++y)
                    ptx::mbar_wait(ring_full + y, ((loads - 1 - y) / 2) & 1, kPPDrainLimitNs, nullptr);
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
    }

    // the sums of the two warpgroups, then of the cluster's CTAs, in that order
    if (warp >= 2) sm_red[128 * ((warp - 2) >> 2) + 32 * (warp & 3) + lane] = sum;
    if (C > 1) {
        ptx::cluster_arrive();
        ptx::cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank == 0 && tid < 128) {
        float w = sm_red[tid] + sm_red[128 + tid];
        for (int r = 1; r < C; ++r) {
            const uint32_t from = ptx::cluster_addr(sm_red + tid, r);
            w += ptx::cluster_ld(from) + ptx::cluster_ld(from + 512);
        }
        const int j = it.j0 + tid;
        // a key past the stream's end may have met anything in its row
        if (j < T) out[(it.b * Hkv + it.hk) * T + j] = j < it.n ? w : 0.f;
    }
    if (C > 1) {  // the other CTAs' sums are read before they leave
        ptx::cluster_arrive();
        ptx::cluster_wait();
    }
}

}  // namespace swa
