// cache.cuh: the budget cache, S slots a key head in no particular order, each with its key and
// value rows, the position it holds and the attention weight that position has received.
// A stream fills slots 0 .. S-1 in order; from then on a new token takes the slot of the
// lightest token that is not among the newest `recent`.
//
// Weights are compared as numbers: -0 equals 0, and NaN counts as +infinity (never lighter
// than a number). Ties go to the lowest slot or position.
#pragma once
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "decode.cuh"
#include "ptx.cuh"

namespace swa {

// Order-preserving image of a weight in 32 unsigned bits.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ------------------------------------------------------------------ append
// One CTA per (b, hk), which reads 12 bytes a slot (weight, position); the loads of kAppendUnroll
// slots a thread are in flight together. 64 streams, 32 heads, 4096 slots, 103 MB: 24 us, 4.3 TB/s
// (0.65 of a copy's rate) on caches that are not in L2: 2048 short CTAs in 2.3 waves, none of which
// has a load in flight while it reduces. Replayed on one set of caches, partly in L2, 21 us (there
// 1, 2 or 8 slots in flight took 24.7, 22.9 and 43.5 us against 20).
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;
__global__ void __launch_bounds__(kAppendThreads, 6)
    cache_append_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v, uint4* __restrict__ kc,
                        uint4* __restrict__ vc, float* __restrict__ wc, int64_t* __restrict__ pc,
                        const int64_t* __restrict__ pos, int64_t* __restrict__ slots, int Hkv, int S, int recent,
                        int vpr, int* status) {
    __shared__ unsigned long long sm_best[32];
    __shared__ int sm_same[32];
    __shared__ int sm_slot;
    const int64_t bh = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nt = blockDim.x;
    const int64_t P = pos[bh / Hkv];
    const uint4 row = tid < vpr ? k[bh * vpr + tid] : tid < 2 * vpr ? v[bh * vpr + tid - vpr] : make_uint4(0, 0, 0, 0);
    float* w = wc + bh * S;
    int64_t* p = pc + bh * S;
    if (P >= S) {
        // the lightest candidate as (weight key, slot), and the slot that holds P already
        unsigned long long best = ~0ull;
        int same = INT32_MAX;
        for (int s0 = tid; s0 < S; s0 += kAppendUnroll * nt) {
            int64_t q[kAppendUnroll];
            float x[kAppendUnroll];
#pragma unroll
            for (int u = 0; u < kAppendUnroll; ++u) {
                const int s = s0 + u * nt;
                q[u] = s < S ? p[s] : INT64_MAX;
                x[u] = s < S ? w[s] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kAppendUnroll; ++u) {
                const int s = s0 + u * nt;
                if (q[u] == P && s < S) same = min(same, s);
                if (q[u] <= P - recent && s < S) {
                    const unsigned long long e = ((unsigned long long)weight_key(x[u]) << 32) | (uint32_t)s;
                    best = e < best ? e : best;
                }
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
            const unsigned long long e = __shfl_xor_sync(0xffffffffu, best, x);
            best = e < best ? e : best;
            same = min(same, __shfl_xor_sync(0xffffffffu, same, x));
        }
        if (lane == 0) {
            sm_best[warp] = best;
            sm_same[warp] = same;
        }
        __syncthreads();
        if (warp == 0) {
            best = lane < nt / 32 ? sm_best[lane] : ~0ull;
            same = lane < nt / 32 ? sm_same[lane] : INT32_MAX;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) {
                const unsigned long long e = __shfl_xor_sync(0xffffffffu, best, x);
                best = e < best ? e : best;
                same = min(same, __shfl_xor_sync(0xffffffffu, same, x));
            }
            if (lane == 0) sm_slot = same != INT32_MAX ? same : best != ~0ull ? (int)(uint32_t)best : -1;
        }
    } else if (tid == 0) {
        sm_slot = P < 0 ? -1 : (int)P;
    }
    __syncthreads();
    const int slot = sm_slot;
    if (tid == 0) {
        slots[bh] = slot;
        if (slot >= 0) {
            w[slot] = 0.f;
            p[slot] = P;
        } else {
            atomicCAS(status, 0, kStatusInvalid);  // a negative position, or no token may leave
        }
    }
    if (slot >= 0 && tid < 2 * vpr) {
        const int e = tid % vpr;
        const int64_t at = (bh * S + slot) * vpr + e;
        if (tid < vpr) kc[at] = row;
        else vc[at] = row;
    }
}

// ------------------------------------------------------------------ seed
// The number of a stream's tokens: T, or lens[b]; -1 (and the status word) if out of range.
__device__ __forceinline__ int stream_len(const int64_t* lens, int64_t b, int T, int* status) {
    if (lens == nullptr) return T;
    const int64_t n = lens[b];
    if (n >= 0 && n <= T) return (int)n;
    atomicCAS(status, 0, kStatusInvalid);
    return -1;
}

constexpr int kSeedThreads = 512;

// A cluster of C CTAs (1 <= C <= 8) per (b, hk) chooses the positions its cache keeps, writes
// them, ascending, with their weights, and copies their rows. The newest `recent` are kept; of
// the older ones the need = S - recent heaviest, found by a radix selection of the weight keys, 11
// bits a pass: the keys above the threshold, and of those equal to it the first few. Each CTA
// counts the digits of its run of positions; the counts meet in distributed shared memory. The
// copy, 4 D bytes read and written a slot, is the bound; the passes over 4 bytes a position come
// before it, each with the latency of its barriers, which is why they are spread over a cluster.
// 32 heads, 16384 positions into 2048 slots, D = 128, 70 MB: 27.7 us on prompts that are not in L2.
// Replayed on one prompt 23, about half of it the selection (there with 8 bits a pass 22.7 against
// 21.6; with C = 1, 2, 4, 8 before the passes could end early 64, 45, 29, 26).
__global__ void __launch_bounds__(kSeedThreads)
    cache_seed_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                      const float* __restrict__ weights, const int64_t* __restrict__ lens, uint4* __restrict__ kc,
                      uint4* __restrict__ vc, float* __restrict__ wc, int64_t* pc, int64_t ksb, int64_t ksh, int64_t kst,
                      int64_t vsb, int64_t vsh, int64_t vst, int Hkv, int T, int S, int recent, int vpr, int C,
                      int* status) {
    constexpr int kWarps = kSeedThreads / 32;
    __shared__ __align__(16) int hist[2][2048];  // of the even and the odd passes
    __shared__ int coarse[2][256];               // of 8 digits each
    __shared__ int all[256];                     // the cluster's coarse counts
    __shared__ int sm_a[kWarps], sm_b[kWarps];
    __shared__ int sm_cta[2];     // this CTA's keys above and equal to the threshold
    __shared__ uint32_t sm_prefix;
    __shared__ int sm_need, sm_found;  // of the keys that share the digits so far: to keep, in all
    const int rank = (int)(blockIdx.x % C);
    const int64_t bh = blockIdx.x / C, b = bh / Hkv, h = bh - b * Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = stream_len(lens, b, T, status);
    const float* w = weights + bh * T;
    float* wo = wc + bh * S;
    int64_t* po = pc + bh * S;
    auto sync = [&] {  // the cluster's CTAs, or this one's threads
        if (C > 1) {
            ptx::cluster_arrive();
            ptx::cluster_wait();
        } else {
            __syncthreads();
        }
    };
    if (n > S) {
        const int old = n - recent;  // positions 0 .. old-1 compete for S - recent slots; old > need
        const int run = ((old + C - 1) / C + 31) / 32 * 32;  // this CTA's: c0 .. c1-1
        const int c0 = min(old, rank * run), c1 = min(old, c0 + run);
        int need = S - recent, found = 0;
        uint32_t prefix = 0, mask = 0;
        // until the digits so far single out exactly the keys still needed (mostly after two)
        for (int pass = 0; pass < 3 && found != need; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            int* mine = hist[pass & 1];
            for (int x = tid; x < 2048; x += kSeedThreads) mine[x] = 0;
            __syncthreads();
            for (int j = c0 + tid; j < c1; j += kSeedThreads) {
                const uint32_t key = weight_key(w[j]);
                if ((key & mask) == prefix) atomicAdd(&mine[(key >> shift) & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            int* mine8 = coarse[pass & 1];
            if (tid < 256) {
                const int4 a = *reinterpret_cast<const int4*>(mine + 8 * tid), c = *reinterpret_cast<const int4*>(mine + 8 * tid + 4);
                mine8[tid] = ((a.x + a.y) + (a.z + a.w)) + ((c.x + c.y) + (c.z + c.w));
            }
            sync();
            if (tid < 256) {
                int sum = mine8[tid];
                if (C > 1) {  // the loads of all CTAs' counts in flight together
                    int x[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        x[r] = r < C ? __float_as_int(ptx::cluster_ld(ptx::cluster_addr(&mine8[tid], r))) : 0;
                    sum = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
                }
                all[tid] = sum;
            }
            __syncthreads();
            if (warp == 0) {
                // the 8 digits among which the count from above reaches need ..
                int own[8], sum = 0;  // lane: coarse digits 255 - 8 lane - i
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += own[i] = all[255 - 8 * lane - i];
                int incl = sum;
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, x);
                    if (lane >= x) incl += y;
                }
                int before = incl - sum, digit = 0;
                const bool mine_ = before < need && need <= incl;
                if (mine_) {
                    int i = 0;
                    while (before + own[i] < need) before += own[i++];
                    digit = 255 - 8 * lane - i;
                }
                const int src = __ffs(__ballot_sync(0xffffffffu, mine_)) - 1;
                before = __shfl_sync(0xffffffffu, before, src);
                digit = __shfl_sync(0xffffffffu, digit, src);
                // .. and the one of them: lane: digit 8 digit + lane % 8 of CTAs lane / 8 and 4 more
                const int* at = mine + 8 * digit + (lane & 7);
                int cnt = 0;
                if (C == 1) {
                    if (lane < 8) cnt = *at;
                } else {
                    const int r = lane >> 3;
                    if (r < C) cnt = __float_as_int(ptx::cluster_ld(ptx::cluster_addr(at, r)));
                    if (r + 4 < C) cnt += __float_as_int(ptx::cluster_ld(ptx::cluster_addr(at, r + 4)));
                }
                cnt += __shfl_xor_sync(0xffffffffu, cnt, 8);
                cnt += __shfl_xor_sync(0xffffffffu, cnt, 16);
                int upto = cnt;  // of this digit and the higher ones of the 8
#pragma unroll
                for (int x = 1; x < 8; x <<= 1) {
                    const int y = __shfl_down_sync(0xffffffffu, upto, x, 8);
                    if ((lane & 7) + x < 8) upto += y;
                }
                before += upto - cnt;
                if (lane < 8 && before < need && need <= before + cnt) {
                    sm_prefix = prefix | ((uint32_t)(8 * digit + lane) << shift);
                    sm_need = need - before;
                    sm_found = cnt;
                }
            }
            __syncthreads();
            prefix = sm_prefix;
            need = sm_need;
            found = sm_found;
            mask = 0xFFFFFFFFu << shift;
            // The next pass clears the other histogram: every CTA has read that one, as it has
            // passed this pass's cluster barrier since.
        }
        // Keep keys > prefix in their digits so far and the first `need` equal to it. Each warp takes one run of
        // positions; the counts of the warps and CTAs before it say where its own go.
        const int wrun = ((c1 - c0 + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int j0 = min(c1, c0 + warp * wrun), j1 = min(c1, j0 + wrun);
        int above = 0, equal = 0;
        for (int j = j0 + lane; j - lane < j1; j += 32) {
            const uint32_t key = j < j1 ? weight_key(w[j]) & mask : 0u;
            above += __popc(__ballot_sync(0xffffffffu, j < j1 && key > prefix));
            equal += __popc(__ballot_sync(0xffffffffu, j < j1 && key == prefix));
        }
        if (lane == 0) {
            sm_a[warp] = above;
            sm_b[warp] = equal;
        }
        __syncthreads();
        if (warp == 0) {
            const int a = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm_a[lane] : 0);
            const int b = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm_b[lane] : 0);
            if (lane == 0) {
                sm_cta[0] = a;
                sm_cta[1] = b;
            }
        }
        sync();
        int na = 0, ne = 0;  // kept above and seen equal before this position
        if (lane < rank) {  // lane: CTA `lane` of the cluster
            na = __float_as_int(ptx::cluster_ld(ptx::cluster_addr(&sm_cta[0], lane)));
            ne = __float_as_int(ptx::cluster_ld(ptx::cluster_addr(&sm_cta[1], lane)));
        }
        if (lane < warp) {  // and warp `lane` of this CTA
            na += sm_a[lane];
            ne += sm_b[lane];
        }
        na = __reduce_add_sync(0xffffffffu, na);
        ne = __reduce_add_sync(0xffffffffu, ne);
        const uint32_t below = (1u << lane) - 1u;
        for (int j = j0 + lane; j - lane < j1; j += 32) {
            const float x = j < j1 ? w[j] : 0.f;
            const uint32_t key = weight_key(x) & mask;
            const uint32_t ba = __ballot_sync(0xffffffffu, j < j1 && key > prefix);
            const uint32_t be = __ballot_sync(0xffffffffu, j < j1 && key == prefix);
            const int a = na + __popc(ba & below), e = ne + __popc(be & below);
            if (j < j1 && (key > prefix || (key == prefix && e < need))) {
                const int at = a + min(e, need);
                wo[at] = x;
                po[at] = j;
            }
            na += __popc(ba);
            ne += __popc(be);
        }
        for (int i = rank * kSeedThreads + tid; i < recent; i += C * kSeedThreads) {
            wo[S - recent + i] = w[old + i];
            po[S - recent + i] = old + i;
        }
    } else {
        for (int j = rank * kSeedThreads + tid; j < n; j += C * kSeedThreads) {
            wo[j] = w[j];
            po[j] = j;
        }
    }
    sync();  // every CTA's positions are visible; no CTA reads another's shared memory after this
    const __nv_bfloat16* kb = k + b * ksb + h * ksh;
    const __nv_bfloat16* vb = v + b * vsb + h * vsh;
    const int rows = kSeedThreads / vpr, e = tid % vpr;  // rows of a step; this thread's 16 bytes of a row
    const int kept = min(n, S), part = (kept + C - 1) / C;
    const int s1 = min(kept, (rank + 1) * part);
    constexpr int kUnroll = 4;
    for (int s0 = rank * part + tid / vpr; s0 < s1; s0 += kUnroll * rows) {
        uint4 x[kUnroll], y[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int s = s0 + u * rows;
            if (s >= s1) continue;
            const int64_t j = __ldcg(po + s);
            x[u] = ld_stream_16(kb + j * kst + 8 * e);
            y[u] = ld_stream_16(vb + j * vst + 8 * e);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int s = s0 + u * rows;
            if (s >= s1) continue;
            kc[(bh * S + s) * vpr + e] = x[u];
            vc[(bh * S + s) * vpr + e] = y[u];
        }
    }
}

}  // namespace swa
