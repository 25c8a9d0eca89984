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
// queries that see the tile's keys come in slices of 64 rows (head gh of the group, rows i0 ..),
// two to a stage of 128 columns. Roles:
//   warp 0, lane 0   TMA producer: the key tile, then the query slices through a ring
//   warp 1           TMEM allocation and MMA issue; S^T double buffered (256 columns)
//   warp 2           -lse log2(e) of each stage's columns into shared memory
//   warps 3 .. 10    p = 2^(s c + nlse) and the row sums: warp = (TMEM quarter, slice)
// Bound: one exp a band pair against 2 D tensor-core flops. The special-function unit alone
// would take 2 x the MMA's time at D = 128, so kKwPolyOf8 of each 8 exponentials are computed
// on the FMA pipe (kw_exp2_parts). Two CTAs share an SM (88 registers a thread, 256 TMEM
// columns, about 100 KB of shared memory), so that one's start and end overlap the other's work.
// Few keys and many queries: a cluster of C CTAs splits the slices of one key tile and adds its
// sums in rank order through distributed shared memory.
constexpr int kKwThreads = 352;
constexpr int kKwSlice = 64;     // query rows of a slice
constexpr int kKwStats = 4;      // stages of nlse in shared memory
constexpr int kKwPolyOf8 = 4;    // column pairs of each 8 whose exponentials use the FMA pipe

template <int D>
struct KwCfg {
    static_assert(D == 64 || D == 128, "head dim 64 or 128");
    static constexpr int kBoxBytes = 128 * 128;  // 128 rows x 64 bf16
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kSliceBytes = kTileBytes / 2;
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kRingOff = kTileBytes;
    static constexpr int kNlOff = kRingOff + kStages * kTileBytes;
    static constexpr int kRedOff = kNlOff + kKwStats * 128 * 4;  // [2][128] sums of the two slices
    static constexpr int kBarOff = kRedOff + 2 * 128 * 4;
    // k_full, ring_full[NS], ring_empty[NS], s_full[2], s_read[2], nl_full[4], nl_free[4], drain
    static constexpr int kNumBars = 2 + 2 * kStages + 4 + 2 * kKwStats;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
    static constexpr uint32_t kTmemCols = 256;
};

// 2^z of two values, as p * 2^n with n = round(z) and p = 2^(z - n), |z - n| <= 1/2. p is the
// polynomial of degree 5 that interpolates 2^f at the Chebyshev nodes of [-1/2, 1/2]: off by at
// most 1.1e-7 of it there, 2.4e-7 with fp32 coefficients and steps. z is held in [-126, 128] (2^128 is
// infinity in fp32); NaN stays NaN.
__device__ __forceinline__ float kw_clamp(float z) {
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(z));  // -126
    asm("min.NaN.f32 %0, %0, 0f43000000;" : "+f"(z));  // 128
    return z;
}
__device__ __forceinline__ void kw_exp2_parts(ptx::f32x2 z, ptx::f32x2& p, ptx::f32x2& pow2) {
    const ptx::f32x2 magic = {12582912.f, 12582912.f};  // 1.5 * 2^23: its sum with z ends in round(z)
    z = {kw_clamp(z.x), kw_clamp(z.y)};
    const ptx::f32x2 t = ptx::add2(z, magic);
    const ptx::f32x2 f = ptx::sub2(z, ptx::sub2(t, magic));
    p = {0.00133908633f, 0.00133908633f};
    p = ptx::fma2(p, f, {0.00967603177f, 0.00967603177f});
    p = ptx::fma2(p, f, {0.0555035695f, 0.0555035695f});
    p = ptx::fma2(p, f, {0.240221068f, 0.240221068f});
    p = ptx::fma2(p, f, {0.693147182f, 0.693147182f});
    p = ptx::fma2(p, f, {1.00000012f, 1.00000012f});
    pow2 = {__uint_as_float(__float_as_uint(t.x) * 0x00800000u + 0x3F800000u),
            __uint_as_float(__float_as_uint(t.y) * 0x00800000u + 0x3F800000u)};
}

// What a CTA works on.
struct KwItem {
    int64_t b, hk;
    int j0, n, i_lo, i_hi;  // keys j0 .., queries i_lo .. i_hi
    int per_head;           // slices of one head
    int s0, s1;             // this CTA's slices of the G * per_head
    __device__ __forceinline__ int head(int s) const { return s / per_head; }
    __device__ __forceinline__ int row(int s) const { return i_lo + kKwSlice * (s % per_head); }
};

// Sums of 32 columns of a row: v scores, nl the columns' nlse; EDGE: only columns
// cmin .. cmax count.
template <bool EDGE>
__device__ __forceinline__ void kw_sum32(const uint32_t (&v)[32], const float* nl, float c2, int cmin, int cmax,
                                         ptx::f32x2 (&acc)[2]) {
    const ptx::f32x2 cc = {c2, c2};
#pragma unroll
    for (int t = 0; t < 32; t += 4) {
        const float4 n4 = *reinterpret_cast<const float4*>(nl + t);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int x = t + 2 * u;
            ptx::f32x2 z = ptx::fma2({__uint_as_float(v[x]), __uint_as_float(v[x + 1])}, cc,
                                     u ? ptx::f32x2{n4.z, n4.w} : ptx::f32x2{n4.x, n4.y});
            const bool in0 = !EDGE || (x >= cmin && x <= cmax), in1 = !EDGE || (x + 1 >= cmin && x + 1 <= cmax);
            if (!EDGE && (x / 2) % 8 % 2 == 0 && (x / 2) % 8 / 2 < kKwPolyOf8) {
                ptx::f32x2 p, e;
                kw_exp2_parts(z, p, e);
                acc[u] = ptx::fma2(p, e, acc[u]);
            } else {
                const ptx::f32x2 p = {ptx::ex2(z.x), ptx::ex2(z.y)};
                acc[u] = ptx::add2(acc[u], {in0 ? p.x : 0.f, in1 ? p.y : 0.f});
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kKwThreads, 2)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const float* __restrict__ lse, const int64_t* __restrict__ lens, float* __restrict__ out,
                          int H, int Hkv, int T, int W, int last, float c2, int C, uint64_t wait_limit_ns, int* status) {
    using Cf = KwCfg<D>;
    constexpr int NS = Cf::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Cf::kBarOff);
    uint64_t* ring_full = k_full + 1;        // [NS]
    uint64_t* ring_empty = ring_full + NS;   // [NS]
    uint64_t* s_full = ring_empty + NS;      // [2]
    uint64_t* s_read = s_full + 2;           // [2] the scores of a buffer are in registers
    uint64_t* nl_full = s_read + 2;          // [kKwStats]
    uint64_t* nl_free = nl_full + kKwStats;  // [kKwStats]
    uint64_t* drain = nl_free + kKwStats;
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
        it.i_hi = (int)min((int64_t)it.n - 1, (int64_t)it.j0 + 127 + W - 1);
        const int rows = it.j0 < it.n ? it.i_hi - it.i_lo + 1 : 0;
        it.per_head = rows > 0 ? (rows + kKwSlice - 1) / kKwSlice : 0;
        const int64_t all = (int64_t)it.per_head * (H / Hkv);
        it.s0 = (int)(all * rank / C);
        it.s1 = (int)(all * (rank + 1) / C);
    }
    const int slices = it.s1 - it.s0, stages = (slices + 1) / 2;
    float sum = 0.f;  // element-wise threads: the sum of this thread's row over its slices

    if (slices > 0) {  // uniform in the CTA
        if (tid == 0) {
            ptx::mbar_init(k_full, 1);
            for (int s = 0; s < NS; ++s) {
                ptx::mbar_init(ring_full + s, 1);
                ptx::mbar_init(ring_empty + s, 1);
            }
            for (int x = 0; x < 2; ++x) {
                ptx::mbar_init(s_full + x, 1);
                ptx::mbar_init(s_read + x, 8);
            }
            for (int x = 0; x < kKwStats; ++x) {
                ptx::mbar_init(nl_full + x, 1);
                ptx::mbar_init(nl_free + x, 8);
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
        uint32_t loads = 0;  // producer: ring stages issued

        if (warp == 0) {
            if (lane == 0) {
                // ------------------------------------------------------------ producer
                bool ok = true;
                ptx::mbar_arrive_expect_tx(k_full, Cf::kTileBytes);
                for (int c = 0; c < D / 64; ++c)
                    ptx::tma_load_4d(smem + c * Cf::kBoxBytes, &tm_k, k_full, 64 * c, it.j0, (int)it.hk, (int)it.b);
                for (int j = 0; j < stages && ok; ++j) {
                    const uint32_t st = loads % NS;
                    if (loads >= (uint32_t)NS)
                        ok = ptx::mbar_wait(ring_empty + st, ((loads / NS) - 1) & 1, wait_limit_ns, abort_flag);
                    if (!ok) break;
                    uint8_t* dst = smem + Cf::kRingOff + st * Cf::kTileBytes;
                    const int here = min(2, slices - 2 * j);
                    ptx::mbar_arrive_expect_tx(ring_full + st, here * Cf::kSliceBytes);
                    for (int x = 0; x < here; ++x) {
                        const int s = it.s0 + 2 * j + x;
                        for (int c = 0; c < D / 64; ++c)
                            ptx::tma_load_4d(dst + c * Cf::kBoxBytes + x * (Cf::kBoxBytes / 2), &tm_q, ring_full + st,
                                             64 * c, it.row(s), (int)it.hk * (H / Hkv) + it.head(s), (int)it.b);
                    }
                    ++loads;
                }
                if (!ok) {
                    atomicCAS(status, 0, 5);
                    *abort_flag = 1;
                }
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
                const uint32_t st = j % NS, buf = j & 1;
                if (j >= 2) ok = wait(s_read + buf, ((j >> 1) - 1) & 1);
                if (ok) ok = wait(ring_full + st, (j / NS) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t q_lo = ((ptx::smem_u32(smem + Cf::kRingOff) + st * Cf::kTileBytes) >> 4) | lo;
                const uint32_t idesc = umma::idesc_bf16_f32(128, slices - 2 * j >= 2 ? 128 : 64, 0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * Cf::kBoxBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_ss_one(tmem + 128 * buf, desc_hi | (k_lo + off), desc_hi | (q_lo + off), idesc,
                                    kk > 0 ? 1u : 0u);
                }
                ptx::tc_commit_one(s_full + buf);
                ptx::tc_commit_one(ring_empty + st);
            }
            if (!ok && lane == 0) {
                atomicCAS(status, 0, 5);
                *abort_flag = 1;
            }
        } else if (warp == 2) {
            // ---------------------------------------------------------------- nlse
            // the loads of a stage are issued two stages before they are stored
            bool ok = true;
            float a[2][4];
            auto fetch = [&](int j, float (&r)[4]) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int s = it.s0 + 2 * j + (x >> 1);
                    r[x] = INFINITY;
                    if (s < it.s1) {
                        const int i = it.row(s) + 32 * (x & 1) + lane;
                        if (i <= it.i_hi)
                            r[x] = lse[((int64_t)it.b * H + it.hk * (H / Hkv) + it.head(s)) * T + i];
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
                    const int st = j % kKwStats;
                    if (j >= kKwStats)
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(nl_free + st, ((j / kKwStats) - 1) & 1, wait_limit_ns,
                                                                    abort_flag));
                    if (!ok) break;
#pragma unroll
                    for (int x = 0; x < 4; ++x) sm_nl[128 * st + 32 * x + lane] = a[y][x] * -1.4426950408889634f;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(nl_full + st);
                    fetch(j + 2, a[y]);
                }
            }
            if (!ok && lane == 0) {
                atomicCAS(status, 0, 5);
                *abort_flag = 1;
            }
        } else {
            // ---------------------------------------------------------------- exponentials, sums
            const int quarter = warp & 3, half = (warp - 3) >> 2;
            const int row = 32 * quarter + lane, jk = it.j0 + row;
            const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16) + 64 * half;
            ptx::f32x2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
            bool ok = true;
            for (int j = 0; j < stages; ++j) {
                const int buf = j & 1, st = j % kKwStats;
                ok = ptx::mbar_wait(s_full + buf, (j >> 1) & 1, wait_limit_ns, abort_flag) &&
                     ptx::mbar_wait(nl_full + st, (j / kKwStats) & 1, wait_limit_ns, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const int s = it.s0 + 2 * j + half;
                const bool have = s < it.s1;  // uniform in the warp
                const int i0 = have ? it.row(s) : 0;
                // columns of this slice that see this thread's key
                const int cmin = jk - i0, cmax = min((int)min((int64_t)jk + W - 1, (int64_t)it.i_hi) - i0, kKwSlice - 1);
                const bool full = i0 >= it.j0 + 127 && (int64_t)i0 + 63 <= (int64_t)it.j0 + W - 1 && i0 + 63 <= it.i_hi;
                const float* nl = sm_nl + 128 * st + 64 * half;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t v[32];
                    if (have) {
                        ptx::tmem_ld32(tl + 128 * buf + 32 * x, v);
                        ptx::tmem_ld_wait();
                        ptx::reg_fence(v);
                    }
                    if (x == 1) {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(s_read + buf);
                    }
                    if (have) {
                        if (full) kw_sum32<false>(v, nl + 32 * x, c2, 0, 31, acc);
                        else kw_sum32<true>(v, nl + 32 * x, c2, cmin - 32 * x, cmax - 32 * x, acc);
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(nl_free + st);
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
                for (uint32_t st = 0; st < (uint32_t)NS && st < loads; ++st) {
                    const uint32_t t = st + ((loads - 1 - st) / NS) * NS;
                    ptx::mbar_wait(ring_full + st, (t / NS) & 1, kPPDrainLimitNs, nullptr);
                }
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

    // the sums of the two slices' threads, then of the cluster's CTAs, in that order
    if (warp >= 3) sm_red[128 * ((warp - 3) >> 2) + 32 * (warp & 3) + lane] = sum;
    if (C > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    if (rank == 0 && tid < 128) {
        float w = sm_red[tid] + sm_red[128 + tid];
        for (int r = 1; r < C; ++r) {
            float x, y;
            uint32_t at;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(sm_red + tid)), "r"(r));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(at + 512));
            w += x + y;
        }
        const int j = it.j0 + tid;
        // a key past the stream's end may have met anything in its row
        if (j < T) out[(it.b * Hkv + it.hk) * T + j] = j < it.n ? w : 0.f;
    }
    if (C > 1) asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

}  // namespace swa
