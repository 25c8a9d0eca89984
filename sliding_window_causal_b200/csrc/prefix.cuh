// prefix.cuh: the queries of a whole batch over a prefix that they share, bf16, D = 64/128, on
// the tensor cores. Row r of key head hk is query head hk G + r % G of stream r / G; every row
// sees every prefix key, so this is a dense attention of B G rows a key head whose softmax is
// taken in splits of the keys and joined by stream_kernel or finish_kernel (attend.cuh): each
// split writes
//   m, l = sum_j 2^(z_j - m), o = sum_j 2^(z_j - m) v_j,   z = scale log2(e) q.k.
//
// prefix_kernel<D, PAIR>: CTA = (key head, group of rows, split of the key tiles), two lanes of
// work x = 0, 1, each with a 128-row tile, its S/P columns (128 x) and O columns (256 + 128 x)
// of TMEM and its softmax warpgroup:
//   PAIR   (more than 128 rows a key head) lane x has row tile x and takes every key tile, so
//          that a key tile in shared memory serves 256 rows;
//   !PAIR  (fewer) both lanes have the one row tile and take every second key tile, and join at
//          the end: with up to 128 rows the prefix's bytes bound the call, and one lane's chain
//          S -> softmax -> P V would be too slow to ask for them.
// While one lane is in its softmax the tensor core works for the other. Roles: warp 0 TMA
// producer (K and V tiles through one ring), warp 1 MMA issuer, warps 4 .. 7 and 8 .. 11 the
// softmax of lanes 0 and 1 (prefix_tile, a row a thread). Q goes to shared memory by plain loads,
// in the layout of a TMA tile, since G query heads of 128 / G streams are no box for every G.
//
// Measured, D = 128: 128 streams of 32 heads, 4 to a key head, behind 65536 keys (PAIR, 137 GFLOP):
// 0.152 ms (0.165 where few keys dominate the rows), 0.9 PFLOP/s of the formula, 1.36 of the products
// issued; P handed over in 1 or 4 parts instead of 2 0.157 and 0.154. What bounds it is a lane's
// chain product, softmax, product, of which two lanes hide only a part (tensor pipe 0.52 busy). 64
// streams of 32 heads (!PAIR): 67 us more for 24576 more keys, 6.0 TB/s.
//
// P is carried as hi + lo bf16 parts (2^-16 of a weight), so that the output is rounded once, as in
// the streams' kernels, and a stream's precision does not depend on how many rows share the prefix.
// !PAIR has room for the second product; in PAIR it lengthens the chain. Of one part only, there
// 0.125 ms, a key that holds much of a row's weight is off by up to 2^-8 of itself: for queries
// scaled by 8 a float64 model of the roundings gives 0.020 on outputs below 4 (0.011 if divided by
// the sum of the rounded weights) where two parts give 0.0078, the output's own rounding. Two parts
// only in the tiles of such keys: 0.133 ms for even rows, but 0.225 for those.
#pragma once
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "attend.cuh"
#include "prefill_pp.cuh"
#include "ptx.cuh"
#include "umma.h"

namespace swa {

constexpr int kPrefixThreads = 384;

template <int D, bool PAIR>
struct PrefixCfg {
    static_assert(D == 64 || D == 128, "head dim 64 or 128");
    static constexpr int kBoxBytes = 128 * 128;
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kQTiles = PAIR ? 2 : 1;
    static constexpr int kStages = (D == 128 ? 7 : 14) - kQTiles;
    static constexpr int kRingOff = kQTiles * kTileBytes;
    static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
    // q_full, ring_full[S], ring_empty[S], s_full[2], p_full[2][kPPParts], o_final[2], drain
    static constexpr int kNumBars = 1 + 2 * kStages + 2 + 2 * kPPParts + 2 + 1;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
    static constexpr uint32_t kTmemCols = 512;
    __device__ static constexpr uint32_t colS(int x) { return 128u * x; }
    __device__ static constexpr uint32_t colO(int x) { return 256u + 128u * x; }
};

// One tile of one row: the thread's 128 scores at TMEM column scol become P = 2^(z - m), z = s c
// (c = scale_log2), in place as bf16 pairs: keys 32k .. 32k+31 in columns 32k .. 32k+15 and the
// rest p - bf16(p), again bf16, in columns 32k+16 .. 32k+31. TAIL: only columns 0 .. last are
// keys. m is the row's reference (-inf before its first tile): a row whose maximum passes it by
// more than 2^8 moves it up by a whole power of two, which rescales O (at ocol) and l exactly.
// after_part(p): part p of P is stored, with one more chunk's arithmetic behind it.
template <int D, bool TAIL, typename AfterPart>
__device__ __forceinline__ void prefix_tile(uint32_t scol, uint32_t ocol, float scale_log2, float& m, float& l, int last,
                                            AfterPart after_part) {
    uint32_t v[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) ptx::tmem_ld32(scol + 32 * c, v[c]);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 4; ++c) ptx::reg_fence(v[c]);
    if (TAIL) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < 32; ++t)
                if (32 * c + t > last) v[c][t] = __float_as_uint(-INFINITY);
    }
    float q[8];  // independent chains of maxima
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = -INFINITY;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < 32; t += 16)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = ptx::max3(q[j], __uint_as_float(v[c][t + 2 * j]), __uint_as_float(v[c][t + 2 * j + 1]));
    const float tm = ptx::max3(ptx::max3(q[0], q[1], q[2]), ptx::max3(q[3], q[4], q[5]), fmaxf(q[6], q[7])) * scale_log2;
    const bool need = m != -INFINITY && tm > m + kPPRescaleThreshold;
    if (__any_sync(0xffffffffu, need)) {
        // in full, so that no weight of this tile exceeds 1; beyond 2^-126 the old sums vanish and
        // the tile's maximum itself is the reference
        const float up = need ? ceilf(tm - m) : 0.f;
        const bool gone = up > 126.f;
        const float f = gone ? 0.f : pp_pow2_neg((int)up);
        __syncwarp();
        pp_rescale<D, false>(ocol, scol, 0, f);
        l *= f;
        m = gone ? tm : m + up;
    }
    if (m == -INFINITY) m = tm;
    const float mu = m == -INFINITY ? 0.f : m;
    const ptx::f32x2 sc = {scale_log2, scale_log2}, nm = {-mu, -mu};
    ptx::f32x2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t ph[16], pl[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const ptx::f32x2 z = ptx::fma2({__uint_as_float(v[c][2 * t]), __uint_as_float(v[c][2 * t + 1])}, sc, nm);
            const ptx::f32x2 e = {ptx::ex2(z.x), ptx::ex2(z.y)};
            acc[t & 1] = ptx::add2(acc[t & 1], e);
            ph[t] = ptx::pack_bf16x2(e.x, e.y);
            const ptx::f32x2 r = ptx::sub2(e, {ptx::bf16lo_f32(ph[t]), ptx::bf16hi_f32(ph[t])});
            pl[t] = ptx::pack_bf16x2(r.x, r.y);
        }
        if (c > 0 && c % (4 / kPPParts) == 0) after_part(c / (4 / kPPParts) - 1);
        ptx::tmem_st16(scol + 32 * c, ph);
        ptx::tmem_st16(scol + 32 * c + 16, pl);
    }
    after_part(kPPParts - 1);
    l += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
}

// a: q, ml, o, B, H, Hkv, G, S (prefix length), chunk (key tiles a split takes), NS, scale_log2
// and status are read. Split s writes the partial states of index s.
template <int D, bool PAIR>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttendArgs a,
                  uint64_t wait_limit_ns) {
    using Cf = PrefixCfg<D, PAIR>;
    constexpr int NS = Cf::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Cf::kBarOff);
    uint64_t* ring_full = q_full + 1;         // [NS]
    uint64_t* ring_empty = ring_full + NS;    // [NS]
    uint64_t* s_full = ring_empty + NS;       // [2]
    uint64_t* p_full = s_full + 2;            // [2][kPPParts]
    uint64_t* o_final = p_full + 2 * kPPParts;  // [2]
    uint64_t* drain = o_final + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cf::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cf::kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int n_rows = a.B * a.G;
    constexpr int kRows = PAIR ? 256 : 128;
    const int groups = (n_rows + kRows - 1) / kRows;
    const int hk = (int)blockIdx.x / groups, row0 = ((int)blockIdx.x % groups) * kRows;
    const int t0 = (int)blockIdx.y * a.chunk, tiles = (a.S + 127) / 128;
    const int n = min(a.chunk, tiles - t0);  // key tiles of this CTA, at least 1
    ptx::launch_dependents();

    if (threadIdx.x == 0) {
        ptx::mbar_init(q_full, 4 * Cf::kQTiles);
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(ring_full + s, 1);
            ptx::mbar_init(ring_empty + s, 1);
        }
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(s_full + x, 1);
            for (int p = 0; p < kPPParts; ++p) ptx::mbar_init(p_full + kPPParts * x + p, 4);
            ptx::mbar_init(o_final + x, 1);
        }
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, Cf::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint32_t loads = 0;  // producer: tiles issued
    // The ring takes the tiles in the order in which the tensor core does, so that none waits for
    // room behind one that is not needed yet: PAIR K0 V0 K1 V1 .., !PAIR K0 K1 V0 K2 V1 K3 ..
    auto pos_k = [&](int t) -> uint32_t { return PAIR ? 2 * t : t == 0 ? 0 : 2 * t - 1; };
    auto pos_v = [&](int t) -> uint32_t { return PAIR || t == n - 1 ? 2 * t + 1 : 2 * t + 2; };
    // the tile at position L of 2 n: t for K_t, ~t for V_t
    auto key_tile = [](int L, int n) -> int {
        if (PAIR) return L & 1 ? ~(L >> 1) : L >> 1;
        if (L == 2 * n - 1) return ~(n - 1);
        return L < 2 ? L : L & 1 ? (L + 1) >> 1 : ~((L - 2) >> 1);
    };

    if (warp < 4) {
        ptx::regs_dec<kPPRoleRegs>();
        if (warp == 0) {
            if (lane == 0) {
                // ------------------------------------------------------------ producer
                bool ok = true;
                for (int L = 0; L < 2 * n && ok; ++L) {
                    const int kt = key_tile(L, n);
                    const bool is_v = kt < 0;
                    const uint32_t st = loads % NS;
                    if (loads >= (uint32_t)NS)
                        ok = ptx::mbar_wait(ring_empty + st, ((loads / NS) - 1) & 1, wait_limit_ns, abort_flag);
                    if (!ok) break;
                    uint8_t* dst = smem + Cf::kRingOff + st * Cf::kTileBytes;
                    ptx::mbar_arrive_expect_tx(ring_full + st, Cf::kTileBytes);
                    for (int c = 0; c < D / 64; ++c)
                        ptx::tma_load_4d(dst + c * Cf::kBoxBytes, is_v ? &tm_v : &tm_k, ring_full + st, 64 * c,
                                         128 * (t0 + (is_v ? ~kt : kt)), hk, 0);
                    ++loads;
                }
                if (!ok) {
                    atomicCAS(a.status, 0, 5);
                    *abort_flag = 1;
                }
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issuer
            const uint32_t idesc_s = umma::idesc_bf16_f32(128, 128, 0);
            const uint32_t idesc_o = umma::idesc_bf16_f32(128, D, 1);
            const uint64_t desc_hi = umma::smem_desc(0, 0, 1024) & 0xFFFFFFFF00000000ull;
            const uint32_t lo_k = (uint32_t)umma::smem_desc(0, 16, 1024);
            const uint32_t lo_v = (uint32_t)umma::smem_desc(0, Cf::kBoxBytes, 1024);
            const uint32_t q_lo = (ptx::smem_u32(smem) >> 4) | lo_k;
            const uint32_t ring_lo = ptx::smem_u32(smem + Cf::kRingOff) >> 4;
            constexpr uint32_t kTileLo = Cf::kTileBytes >> 4;
            bool ok = pp_wait_warp(q_full, 0, wait_limit_ns, abort_flag);
            auto arrived = [&](uint32_t L) {
                if (ok) ok = pp_wait_warp(ring_full + L % NS, (L / NS) & 1, wait_limit_ns, abort_flag);
            };
            auto issue_s = [&](int x, uint32_t L) {  // S_x = Q K^T, K the L-th tile of the ring
                ptx::tc_fence_after();
                const uint32_t k_lo = (ring_lo + L % NS * kTileLo) | lo_k;
                const uint32_t a_lo = q_lo + (PAIR ? x * kTileLo : 0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * Cf::kBoxBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_ss_one(tmem + Cf::colS(x), desc_hi | (a_lo + off), desc_hi | (k_lo + off), idesc_s,
                                    kk > 0 ? 1u : 0u);
                }
                ptx::tc_commit_one(s_full + x);
            };
            auto issue_pv = [&](int x, uint32_t L, int j) {  // O_x (+)= P_x V as the parts of P arrive
                const uint32_t v_lo = (ring_lo + L % NS * kTileLo) | lo_v;
#pragma unroll
                for (int part = 0; part < kPPParts; ++part) {
                    if (ok) ok = pp_wait_warp(p_full + kPPParts * x + part, j & 1, wait_limit_ns, abort_flag);
                    if (!ok) return;
                    ptx::tc_fence_after();
                    constexpr int kPer = 8 / kPPParts;
#pragma unroll
                    for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                        for (int kk = part * kPer; kk < (part + 1) * kPer; ++kk)
                            ptx::mma_ts_one(tmem + Cf::colO(x), tmem + Cf::colS(x) + pp_pcol(kk) + 16 * lo,
                                            desc_hi | (v_lo + kk * (2048 >> 4)), idesc_o,
                                            (j > 0 || kk > 0 || lo > 0) ? 1u : 0u);
                }
            };
            if (PAIR) {
                arrived(0);
                if (ok) {
                    issue_s(0, 0);
                    issue_s(1, 0);
                    ptx::tc_commit_one(ring_empty + 0);
                }
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t Lv = pos_v(j), Lk = pos_k(j + 1);
                    arrived(Lv);
                    if (j + 1 < n) arrived(Lk);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (ok) issue_pv(x, Lv, j);
                        if (!ok) break;
                        if (j + 1 < n) issue_s(x, Lk);  // after P_x V in the tensor core's order: P_x is read
                        else ptx::tc_commit_one(o_final + x);
                    }
                    if (!ok) break;
                    ptx::tc_commit_one(ring_empty + Lv % NS);
                    if (j + 1 < n) ptx::tc_commit_one(ring_empty + Lk % NS);
                }
            } else {
                for (int t = 0; t < 2 && t < n && ok; ++t) {
                    arrived(pos_k(t));
                    if (!ok) break;
                    issue_s(t, pos_k(t));
                    ptx::tc_commit_one(ring_empty + pos_k(t) % NS);
                }
                for (int t = 0; t < n && ok; ++t) {
                    const int x = t & 1;
                    const uint32_t Lv = pos_v(t), Lk = pos_k(t + 2);
                    arrived(Lv);
                    if (ok) issue_pv(x, Lv, t >> 1);
                    if (!ok) break;
                    ptx::tc_commit_one(ring_empty + Lv % NS);
                    if (t + 2 < n) {
                        arrived(Lk);
                        if (!ok) break;
                        issue_s(x, Lk);
                        ptx::tc_commit_one(ring_empty + Lk % NS);
                    } else {
                        ptx::tc_commit_one(o_final + x);
                    }
                }
            }
            if (!ok && lane == 0) {
                atomicCAS(a.status, 0, 5);
                *abort_flag = 1;
            }
        }
    } else {
        // -------------------------------------------------------------------- softmax
        ptx::regs_inc<kPPSoftmaxRegs>();
        const int x = (warp - 4) >> 2, quarter = warp & 3;
        const int row = 32 * quarter + lane;
        const int r = row0 + (PAIR ? 128 * x : 0) + row;
        const bool live = r < n_rows;
        const int64_t qrow = live ? (int64_t)(r / a.G) * a.H + hk * a.G + r % a.G : 0;
        if (PAIR || x == 0) {
            // this thread's query row, as TMA with 128-byte swizzle would place it
            uint8_t* dst = smem + (PAIR ? x * Cf::kTileBytes : 0) + row * 128;
            const uint4* src = reinterpret_cast<const uint4*>(a.q + qrow * D);
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
                *reinterpret_cast<uint4*>(dst + (e >> 3) * Cf::kBoxBytes + (((e & 7) ^ (row & 7)) << 4)) =
                    live ? src[e] : make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(q_full);
        }
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t scol = tl + Cf::colS(x), ocol = tl + Cf::colO(x);
        const int mine = PAIR ? n : (n + 1 - x) / 2;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        // S_x(j) follows P_x(j-1) V in the tensor core's order: once S_x(j) is there, O_x is at rest
        auto after_part = [&](int part) {
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(p_full + kPPParts * x + part);
        };
        for (int j = 0; j < mine; ++j) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full + x, j & 1, wait_limit_ns, abort_flag));
            if (!ok) break;
            ptx::tc_fence_after();
            const int last = a.S - 1 - 128 * (t0 + (PAIR ? j : 2 * j + x));  // last key of the tile
            if (last >= 127) prefix_tile<D, false>(scol, ocol, a.scale_log2, m, l, 127, after_part);
            else prefix_tile<D, true>(scol, ocol, a.scale_log2, m, l, last, after_part);
        }
        const int64_t at = qrow * a.NS + (int)blockIdx.y;
        if (PAIR) {
            if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(o_final + x, 0, wait_limit_ns, abort_flag));
            if (ok) {
                ptx::tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    ptx::tmem_ld32(ocol + 32 * c, o);
                    ptx::tmem_ld_wait();
                    ptx::reg_fence(o);
                    if (live) {
                        float4* to = reinterpret_cast<float4*>(a.o + at * D + 32 * c);
#pragma unroll
                        for (int t = 0; t < 8; ++t)
                            to[t] = make_float4(__uint_as_float(o[4 * t]), __uint_as_float(o[4 * t + 1]),
                                                __uint_as_float(o[4 * t + 2]), __uint_as_float(o[4 * t + 3]));
                    }
                }
            }
            if (live) a.ml[at] = make_float2(m, l);
        } else {
            // The two lanes' states of a row become one: O_0 and O_1 are in the same TMEM lanes, so
            // each warpgroup joins half of the columns; m and l cross through shared memory (the
            // ring's first bytes: its tiles are read once both lanes' O is final).
            for (int y = 0; y < 2 && y < n; ++y)
                if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(o_final + y, 0, wait_limit_ns, abort_flag));
            float2* sm_ml = reinterpret_cast<float2*>(smem + Cf::kRingOff);  // [2][128]
            if (ok) sm_ml[128 * x + row] = make_float2(m, l);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (ok) {
                ptx::tc_fence_after();
                const float2 other = sm_ml[128 * (1 - x) + row];
                const float M = fmaxf(m, other.x);
                const float mine_f = m == -INFINITY ? 0.f : ptx::ex2(m - M);
                const float other_f = other.x == -INFINITY ? 0.f : ptx::ex2(other.x - M);
                const float f0 = x ? other_f : mine_f, f1 = x ? mine_f : other_f;
#pragma unroll 1
                for (int c = x * (D / 64); c < (x + 1) * (D / 64); ++c) {
                    uint32_t o[2][32];
                    ptx::tmem_ld32(tl + Cf::colO(0) + 32 * c, o[0]);
                    ptx::tmem_ld32(tl + Cf::colO(1) + 32 * c, o[1]);
                    ptx::tmem_ld_wait();
                    ptx::reg_fence(o[0]);
                    ptx::reg_fence(o[1]);
                    if (live) {
                        float4* to = reinterpret_cast<float4*>(a.o + at * D + 32 * c);
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            float v[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // with one key tile O_1 was never written
                                const float o1 = n > 1 ? __uint_as_float(o[1][4 * t + e]) * f1 : 0.f;
                                v[e] = fmaf(__uint_as_float(o[0][4 * t + e]), f0, o1);
                            }
                            to[t] = make_float4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
                if (live && x == 0) a.ml[at] = make_float2(M, fmaf(l, f0, other.y * f1));
            }
        }
        if (!ok) {
            atomicCAS(a.status, 0, 5);
            *abort_flag = 1;
        }
    }

    // ------------------------------------------------------------------------ teardown
    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        if (warp == 0 && lane == 0) {
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

}  // namespace swa
