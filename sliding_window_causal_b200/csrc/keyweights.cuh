// keyweights.cuh: the attention weight that each key of a prompt received,
//   w[b,hk,j] = sum over the G query heads of hk, sum over queries i of the counted rows whose
//               band holds j, of exp(scale q_i . k_j - lse_i),
// from the log-sum-exp that the training forward writes. The rows counted are the last
// `last` of the stream's n tokens: max(0, n - last) <= i < n. Keys at or past n get 0.
//
// key_weights_simt_kernel: fp32 FMA on 64-key x 64-query score tiles, for fp32 inputs. One CTA
// owns 64 keys and runs over the query tiles and heads that see them, so every sum has one
// owner and a fixed order.
#pragma once
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "cache.cuh"
#include "decode.cuh"

namespace swa {

constexpr int kKwTile = 64;   // keys and queries of a score tile
constexpr int kKwDepth = 32;  // head columns staged at a time

template <typename TIn>
__global__ void __launch_bounds__(256)
    key_weights_simt_kernel(const TIn* __restrict__ q, const TIn* __restrict__ k, const float* __restrict__ lse,
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
            const TIn* qb = q + b * qsb + h * qsh;
            const TIn* kb = k + b * ksb + hk * ksh;
            for (int i0 = i_lo; i0 <= i_hi; i0 += kKwTile) {
                float c[4][4] = {};
                for (int d0 = 0; d0 < D; d0 += kKwDepth) {
                    __syncthreads();
                    for (int x = tid; x < kKwTile * kKwDepth; x += 256) {
                        const int r = x / kKwDepth, d = x % kKwDepth;
                        const bool in = d0 + d < D;
                        sq[d][r] = in && i0 + r <= i_hi ? to_f32(qb[(int64_t)(i0 + r) * qst + d0 + d]) : 0.f;
                        sk[d][r] = in && j0 + r < n ? to_f32(kb[(int64_t)(j0 + r) * kst + d0 + d]) : 0.f;
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

}  // namespace swa
