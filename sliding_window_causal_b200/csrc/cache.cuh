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
// One CTA per (b, hk). Bound by the 12 bytes a slot (weight, position) that the choice reads.
__global__ void __launch_bounds__(1024)
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
    float* w = wc + bh * S;
    int64_t* p = pc + bh * S;
    if (P >= S) {
        // the lightest candidate as (weight key, slot), and the slot that holds P already
        unsigned long long best = ~0ull;
        int same = INT32_MAX;
        for (int s = tid; s < S; s += nt) {
            const int64_t q = p[s];
            const float x = w[s];
            if (q == P) same = min(same, s);
            if (q <= P - recent) {
                const unsigned long long e = ((unsigned long long)weight_key(x) << 32) | (uint32_t)s;
                best = e < best ? e : best;
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
        if (tid < vpr) kc[at] = k[bh * vpr + e];
        else vc[at] = v[bh * vpr + e];
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

constexpr int kSeedThreads = 1024;

// One CTA per (b, hk) chooses the positions its cache keeps and writes them, ascending, with
// their weights. The newest `recent` are kept; of the older ones the need = S - recent
// heaviest, found by a radix selection of the weight keys, 8 bits a pass: the keys above the
// threshold, and of those equal to it the first few.
__global__ void __launch_bounds__(kSeedThreads)
    seed_select_kernel(const float* __restrict__ weights, const int64_t* __restrict__ lens, float* __restrict__ wc,
                       int64_t* __restrict__ pc, int Hkv, int T, int S, int recent, int* status) {
    __shared__ int hist[256];
    __shared__ int sm_a[32], sm_b[32];
    __shared__ uint32_t sm_prefix;
    __shared__ int sm_need;
    const int64_t bh = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = stream_len(lens, bh / Hkv, T, status);
    const float* w = weights + bh * T;
    float* wo = wc + bh * S;
    int64_t* po = pc + bh * S;
    if (n <= S) {
        for (int j = tid; j < n; j += kSeedThreads) {
            wo[j] = w[j];
            po[j] = j;
        }
        return;
    }
    const int old = n - recent;  // positions 0 .. old-1 compete for S - recent slots; old > need
    int need = S - recent;
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < old; j += kSeedThreads) {
            const uint32_t key = weight_key(w[j]);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (warp == 0) {  // the digit at which the count from above reaches need
            int own[8], sum = 0;  // lane: digits 255 - 8 lane - i
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += own[i] = hist[255 - 8 * lane - i];
            int incl = sum;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, x);
                if (lane >= x) incl += y;
            }
            int before = incl - sum;
            if (before < need && need <= incl) {
                int i = 0;
                while (before + own[i] < need) before += own[i++];
                sm_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
                sm_need = need - before;
            }
        }
        __syncthreads();
        prefix = sm_prefix;
        need = sm_need;
        __syncthreads();
    }
    // Keep keys > prefix and the first `need` keys equal to it. Each warp takes one run of
    // positions; the counts of the warps before it say where its own go.
    const int run = ((old + 31) / 32 + 31) / 32 * 32;
    const int j0 = min(old, warp * run), j1 = min(old, j0 + run);
    int above = 0, equal = 0;
    for (int j = j0 + lane; j - lane < j1; j += 32) {
        const uint32_t key = j < j1 ? weight_key(w[j]) : 0u;
        above += __popc(__ballot_sync(0xffffffffu, j < j1 && key > prefix));
        equal += __popc(__ballot_sync(0xffffffffu, j < j1 && key == prefix));
    }
    if (lane == 0) {
        sm_a[warp] = above;
        sm_b[warp] = equal;
    }
    __syncthreads();
    int na = 0, ne = 0;  // kept above and seen equal before this position
    for (int x = 0; x < warp; ++x) {
        na += sm_a[x];
        ne += sm_b[x];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int j = j0 + lane; j - lane < j1; j += 32) {
        const float x = j < j1 ? w[j] : 0.f;
        const uint32_t key = weight_key(x);
        const uint32_t ba = __ballot_sync(0xffffffffu, j < j1 && key > prefix);
        const uint32_t be = __ballot_sync(0xffffffffu, j < j1 && key == prefix);
        const int a = na + __popc(ba & below), e = ne + __popc(be & below);
        const bool take = j < j1 && (key > prefix || (key == prefix && e < need));
        if (take) {
            const int at = a + min(e, need);
            wo[at] = x;
            po[at] = j;
        }
        na += __popc(ba);
        ne += __popc(be);
    }
    for (int i = tid; i < recent; i += kSeedThreads) {
        wo[S - recent + i] = w[old + i];
        po[S - recent + i] = old + i;
    }
}

// Copy the kept positions' key and value rows into their slots, 16 bytes a thread.
__global__ void __launch_bounds__(256)
    seed_gather_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                       const int64_t* __restrict__ lens, const int64_t* __restrict__ pc, uint4* __restrict__ kc,
                       uint4* __restrict__ vc, int64_t ksb, int64_t ksh, int64_t kst, int64_t vsb, int64_t vsh,
                       int64_t vst, int Hkv, int T, int S, int vpr, int64_t n_vec) {
    ptx::grid_dependency_wait();
    for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < n_vec; x += (int64_t)gridDim.x * blockDim.x) {
        const int e = (int)(x % vpr);
        const int64_t row = x / vpr;  // bh * S + slot
        const int64_t bh = row / S, b = bh / Hkv, h = bh - b * Hkv;
        const int64_t n = lens == nullptr ? T : lens[b];
        if (n < 0 || n > T || row - bh * S >= n) continue;
        const int64_t j = pc[row];
        kc[x] = *reinterpret_cast<const uint4*>(k + b * ksb + h * ksh + j * kst + 8 * e);
        vc[x] = *reinterpret_cast<const uint4*>(v + b * vsb + h * vsh + j * vst + 8 * e);
    }
}

}  // namespace swa
