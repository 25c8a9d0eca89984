// attend.cuh: one query per stream over keys in memory (a prefix shared by all streams, the
// stream's ring, the stream's budget cache), bf16, D = 64/128, G query heads to a key head.
//
// The softmax of a row is taken in splits of its keys, each an online softmax state
//   m = max_j z_j,  l = sum_j 2^(z_j - m),  o = sum_j 2^(z_j - m) v_j,   z = scale log2(e) q.k,
// and joined: m* = max m, out = sum 2^(m - m*) o / sum 2^(m - m*) l.
//
// A CTA takes some keys for up to 8 queries that share them, so HBM is the bound: 4 D bytes a key
// against 32 D multiply-adds. stream_kernel: a cluster of CTAs finishes a (stream, key head) by
// itself. attend_kernel: any number of splits, when a cluster is too few CTAs for the keys or
// there are more than 8 queries, joined by finish_kernel. The products go through m16n8k16 with
// the keys as the 16 rows (S^T = K Q^T and O^T = V^T P^T), which spends no tile rows on missing
// queries. Every fragment comes straight from 16-byte loads: the order of the head dimension
// inside a product is free as long as K and Q agree (a lane's 16 bytes are two k-steps), and in
// O^T it is the order of the output rows. P crosses from accumulator to operand layout by an 8x8 transpose inside
// the warp. P is carried as two bf16 parts (hi + lo, 16 bits of weight), so that the output
// is rounded once: the products are far from bounding the kernel. m, l, o are fp32; o and l
// are rescaled only when a score passes m by more than 2^8.
#pragma once
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "decode.cuh"
#include "ptx.cuh"

namespace swa {

constexpr int kAttendWarps = 4;
constexpr int kAttendStep = 16 * kAttendWarps;  // slots a CTA takes per step
constexpr int kAttendQueries = 8;               // queries a CTA serves
constexpr float kAttendRescale = 8.f;

// Where a call's queries, keys and partial states are. Row = b * H + h.
struct AttendArgs {
    const __nv_bfloat16* q;    // [B, H, D]
    const __nv_bfloat16* k;    // ring or cache [B, Hkv, S, D]; prefix: (h, t) strides
    const __nv_bfloat16* v;
    const int64_t* pos;        // [B]; not read by prefix_kernel
    float2* ml;                // [B*H][NS] (m, l)
    float* o;                  // [B*H][NS][D]
    float* scores;             // [B*Hkv][G][S] z of every slot, or null
    int64_t k_head, k_row, v_head, v_row;  // element strides
    int B, H, Hkv, G, S;       // S: slots, or the prefix length
    int chunk, split0, NS;     // keys a split takes, first split index, splits in all
    float scale_log2;
    int* status;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The slots that the query at position P sees: none, and a report, if it is negative.
__device__ __forceinline__ int attend_slots(int64_t P, int S, int* status, bool report) {
    if (P >= 0) return P < (int64_t)S ? (int)P + 1 : S;
    if (report) atomicCAS(status, 0, kStatusInvalid);
    return 0;
}
__device__ __forceinline__ uint32_t word(const uint4& u, int w) { return w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w; }

// The online softmax of 8 queries over some keys, as one warp of a CTA holds it: queries 2t and
// 2t+1 of lane (g, t), o in the layout of the accumulators of O^T.
template <int D>
struct AttendState {
    static constexpr int KL = D / 32;  // 16-byte pieces of a key row per lane
    static constexpr int VL = D / 64;  // 16-byte pieces of a value row per lane
    static constexpr int MT = D / 16;  // 16-row tiles of O^T
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[MT][4];
    uint32_t qf[KL][4];  // B fragments of Q^T: query g

    // qr: query g's row, or null
    __device__ __forceinline__ void start(const __nv_bfloat16* qr, int t) {
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const uint4 u = qr ? *reinterpret_cast<const uint4*>(qr + 32 * i + 8 * t) : make_uint4(0, 0, 0, 0);
            qf[i][0] = u.x; qf[i][1] = u.y; qf[i][2] = u.z; qf[i][3] = u.w;
        }
    }

    // Keys r0 .. r1-1 of k, v (row strides k_row, v_row); the CTA's warps take 16 each in turn.
    // put(query, key, z) gets every score.
    template <typename Put>
    __device__ __forceinline__ void keys(const __nv_bfloat16* k, const __nv_bfloat16* v, int64_t k_row, int64_t v_row,
                                         int r0, int r1, float scale_log2, int warp, int g, int t, Put put) {
        const __nv_bfloat16* kb = k + 8 * t;
        const __nv_bfloat16* vb = v + 8 * g;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int base = r0 + 16 * warp; base < r1; base += kAttendStep) {
            uint4 kr[2][KL], vr[4][VL];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int slot = base + g + 8 * x;
#pragma unroll
                for (int i = 0; i < KL; ++i) kr[x][i] = slot < r1 ? ld_stream_16(kb + slot * k_row + 32 * i) : zero;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int slot = base + 2 * t + (x & 1) + 8 * (x >> 1);
#pragma unroll
                for (int i = 0; i < VL; ++i) vr[x][i] = slot < r1 ? ld_stream_16(vb + slot * v_row + 64 * i) : zero;
            }
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                mma_bf16(c, kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, qf[i][0], qf[i][1]);
                mma_bf16(c, kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, qf[i][2], qf[i][3]);
            }
            const bool v0 = base + g < r1, v1 = base + g + 8 < r1;
            const float z0 = v0 ? c[0] * scale_log2 : -INFINITY, z1 = v0 ? c[1] * scale_log2 : -INFINITY;
            const float z2 = v1 ? c[2] * scale_log2 : -INFINITY, z3 = v1 ? c[3] * scale_log2 : -INFINITY;
            if (v0) {
                put(2 * t, base + g, z0);
                put(2 * t + 1, base + g, z1);
            }
            if (v1) {
                put(2 * t, base + g + 8, z2);
                put(2 * t + 1, base + g + 8, z3);
            }
            float t0 = fmaxf(z0, z2), t1 = fmaxf(z1, z3);
            if (__any_sync(0xffffffffu, t0 > m0 + kAttendRescale || t1 > m1 + kAttendRescale)) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
                    t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
                }
                const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
                const float f0 = m0 == -INFINITY ? 0.f : ptx::ex2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[i][0] *= f0;
                    o[i][1] *= f1;
                    o[i][2] *= f0;
                    o[i][3] *= f1;
                }
            }
            const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
            const float p0 = ptx::ex2(z0 - u0), p1 = ptx::ex2(z1 - u1), p2 = ptx::ex2(z2 - u0), p3 = ptx::ex2(z3 - u1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            const uint32_t h01 = ptx::pack_bf16x2(p0, p1), h23 = ptx::pack_bf16x2(p2, p3);
            const uint32_t e01 = ptx::pack_bf16x2(p0 - ptx::bf16lo_f32(h01), p1 - ptx::bf16hi_f32(h01));
            const uint32_t e23 = ptx::pack_bf16x2(p2 - ptx::bf16lo_f32(h23), p3 - ptx::bf16hi_f32(h23));
            const uint32_t bh0 = transpose_8x8(h01), bh1 = transpose_8x8(h23);
            const uint32_t bl0 = transpose_8x8(e01), bl1 = transpose_8x8(e23);
#pragma unroll
            for (int i = 0; i < VL; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t x0 = word(vr[0][i], w), x1 = word(vr[1][i], w), x2 = word(vr[2][i], w), x3 = word(vr[3][i], w);
                    const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
                    const uint32_t a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
                    mma_bf16(o[4 * i + w], a0, a1, a2, a3, bh0, bh1);
                    mma_bf16(o[4 * i + w], a0, a1, a2, a3, bl0, bl1);
                }
        }
    }
};

// The states of a CTA's warps, joined: done(query, d, M, L, A) for every 4 columns d of the
// first nq queries, once each, and may overwrite these columns of o[0].
template <int D>
struct AttendJoin {
    float m[kAttendWarps][kAttendQueries], l[kAttendWarps][kAttendQueries];
    alignas(16) float o[kAttendWarps][kAttendQueries][D + 8];  // read and written 16 bytes at a time
    static_assert((D + 8) * sizeof(float) % 16 == 0, "a row of o starts on 16 bytes");

    template <typename Done>
    __device__ __forceinline__ void run(AttendState<D>& st, int nq, int tid, Done done) {
        const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, x);
            st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, x);
        }
        if (g == 0) {
            m[warp][2 * t] = st.m0;
            m[warp][2 * t + 1] = st.m1;
            l[warp][2 * t] = st.l0;
            l[warp][2 * t + 1] = st.l1;
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int d = 64 * i + 8 * g + 2 * w;
                *reinterpret_cast<float2*>(&o[warp][2 * t][d]) = make_float2(st.o[4 * i + w][0], st.o[4 * i + w][2]);
                *reinterpret_cast<float2*>(&o[warp][2 * t + 1][d]) = make_float2(st.o[4 * i + w][1], st.o[4 * i + w][3]);
            }
        __syncthreads();
        for (int x = tid; x < nq * (D / 4); x += kAttendWarps * 32) {
            const int i = x / (D / 4), d = (x % (D / 4)) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttendWarps; ++w) M = fmaxf(M, m[w][i]);
            float L = 0.f;
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttendWarps; ++w) {
                // a warp without a key has l = 0 and o = 0
                const float f = m[w][i] == -INFINITY ? 0.f : ptx::ex2(m[w][i] - M);
                L = fmaf(l[w][i], f, L);
                const float4 v = *reinterpret_cast<const float4*>(&o[w][i][d]);
                A.x = fmaf(v.x, f, A.x);
                A.y = fmaf(v.y, f, A.y);
                A.z = fmaf(v.z, f, A.z);
                A.w = fmaf(v.w, f, A.w);
            }
            done(i, d, M, L, A);
        }
    }
};

static_assert(alignof(AttendJoin<64>) >= 16 && alignof(AttendJoin<128>) >= 16, "16-byte accesses of o");

// ------------------------------------------------------------------ splits of any number
// CTA = (stream, key head, 8 of its queries, split of the slots 0 .. min(pos+1, S)-1). More than 8
// query heads to a key head read its keys and values once for each 8, mostly from L2: 64 streams of
// 64 heads, 16 to a key head, 4096 slots, D = 128, with weights (545 MB): 144 us and 40 in
// finish_kernel, which reads the scores again; 9 to a key head of 72 (1.09 GB) 271 and 47.
template <int D, bool SCORES>
__global__ void __launch_bounds__(kAttendWarps * 32, D == 128 ? 4 : 6) attend_kernel(const AttendArgs a) {
    __shared__ AttendJoin<D> join;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int s = blockIdx.y;
    const int qtiles = (a.G + kAttendQueries - 1) / kAttendQueries;
    const int64_t unit = blockIdx.x / qtiles, b = unit / a.Hkv;
    const int q0 = (int)(blockIdx.x % qtiles) * kAttendQueries;
    const int nq = min(kAttendQueries, a.G - q0);
    const int64_t row0 = b * a.H + (unit - b * a.Hkv) * a.G + q0;
    const int n = attend_slots(a.pos[b], a.S, a.status, tid == 0 && s == 0);
    const int r0 = s * a.chunk;
    const int r1 = min(r0 + a.chunk, n);
    if (r0 >= r1) {  // nothing of this split is valid
        if (tid < nq) a.ml[(row0 + tid) * a.NS + a.split0 + s] = make_float2(-INFINITY, 0.f);
        return;
    }
    AttendState<D> st;
    st.start(g < nq ? a.q + (row0 + g) * D : nullptr, t);
    float* zrow = SCORES ? a.scores + (unit * a.G + q0) * a.S : nullptr;
    st.keys(a.k + unit * a.k_head, a.v + unit * a.v_head, a.k_row, a.v_row, r0, r1, a.scale_log2, warp, g, t,
            [&](int i, int slot, float z) {
                if (SCORES && i < nq) zrow[(int64_t)i * a.S + slot] = z;
            });
    join.run(st, nq, tid, [&](int i, int d, float M, float L, const float4& A) {
        const int64_t at = (row0 + i) * a.NS + a.split0 + s;
        *reinterpret_cast<float4*>(a.o + at * D + d) = A;
        if (d == 0) a.ml[at] = make_float2(M, L);
    });
}

// ------------------------------------------------------------------ one cluster per key head
// stream_kernel: a cluster of C CTAs takes all keys of one (stream, key head): the first P0 keys
// of the prefix, when it is short enough for every stream to read it by itself, and the slots.
// Its CTAs join their states through distributed shared memory, together with the np partial
// states that a kernel before it has left for the rest of the prefix, write the output rows and,
// SCORES, add the attention weights from the scores they kept in shared memory: no workspace
// but the prefix's, one launch, no traffic beyond the inputs and outputs. G <= 8. 64 streams, 32
// heads, 4096 slots, D = 128, with weights: 643 us, 6.8 TB/s (attend_kernel and finish_kernel,
// which write and read the scores once more: 701 us). Few slots a CTA leave the latency of its
// chain of loads: 1024 (stream, key head)s of 256 slots take 27 us for 134 MB.
struct StreamArgs {
    AttendArgs a;                 // slots; ml, o, NS: the np partial states of a row
    const __nv_bfloat16* pk;      // the prefix: (h, t) strides
    const __nv_bfloat16* pv;
    int64_t pk_head, pk_row, pv_head, pv_row;
    int P0, pchunk;               // prefix keys read here; keys of a CTA
    int C;
    __nv_bfloat16* out;
    float* weights;
};

__device__ __forceinline__ void ldcg_vec(const float* p, float (&v)[4]) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void ldcg_vec(const float* p, float (&v)[2]) {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
    v[0] = x.x; v[1] = x.y;
}

template <int D, bool SCORES>
__global__ void __launch_bounds__(kAttendWarps * 32, D == 128 ? 4 : 6) stream_kernel(const StreamArgs sa) {
    const AttendArgs& a = sa.a;
    __shared__ AttendJoin<D> join;
    __shared__ float sm_m[kAttendQueries], sm_l[kAttendQueries], sm_lse[kAttendQueries];
    extern __shared__ float sm_z[];  // [G][chunk]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int C = sa.C, rank = (int)(blockIdx.x % C);
    const int64_t unit = blockIdx.x / C, b = unit / a.Hkv;
    const int hk = (int)(unit - b * a.Hkv), nq = a.G;
    const int64_t row0 = b * a.H + hk * a.G;
    const int64_t pos = a.pos[b];
    AttendState<D> st;
    st.start(g < nq ? a.q + (row0 + g) * D : nullptr, t);  // beside the load of pos
    const int n = attend_slots(pos, a.S, a.status, tid == 0 && rank == 0);
    const int r0 = min(rank * a.chunk, n), r1 = min(r0 + a.chunk, n);

    if (sa.P0 > 0) {
        const int p0 = min(rank * sa.pchunk, sa.P0), p1 = min(p0 + sa.pchunk, sa.P0);
        st.keys(sa.pk + hk * sa.pk_head, sa.pv + hk * sa.pv_head, sa.pk_row, sa.pv_row, p0, p1, a.scale_log2, warp, g, t,
                [](int, int, float) {});
    }
    st.keys(a.k + unit * a.k_head, a.v + unit * a.v_head, a.k_row, a.v_row, r0, r1, a.scale_log2, warp, g, t,
            [&](int i, int slot, float z) {
                if (SCORES && i < nq) sm_z[i * a.chunk + slot - r0] = z;
            });
    join.run(st, nq, tid, [&](int i, int d, float M, float L, const float4& A) {
        *reinterpret_cast<float4*>(&join.o[0][i][d]) = A;
        if (d == 0) {
            sm_m[i] = M;
            sm_l[i] = L;
        }
    });
    if (C > 1) {
        ptx::cluster_arrive();
        ptx::cluster_wait();
    } else {
        __syncthreads();
    }
    ptx::grid_dependency_wait();  // the prefix's partial states
    for (int i = warp; i < nq; i += kAttendWarps) {  // a warp joins a row
        const int64_t row = row0 + i;
        const float2* ml = a.ml + row * a.NS;
        float cm = -INFINITY, cl = 0.f;  // lane: the state of CTA `lane`
        if (lane < C) {
            cm = ptx::cluster_ld(ptx::cluster_addr(&sm_m[i], lane));
            cl = ptx::cluster_ld(ptx::cluster_addr(&sm_l[i], lane));
        }
        // the prefix's: of a lane, state `lane` of every 32 (the first 32 stay in registers)
        const float2 e0 = lane < a.NS ? __ldcg(ml + lane) : make_float2(-INFINITY, 0.f);
        const bool writes = i % C == rank;  // the output row
        constexpr int E = D / 32;           // its columns E lane ..
        float v[16][E];                     // the prefix's first states, on their way meanwhile
        auto fetch = [&](int s0) {
#pragma unroll
            for (int y = 0; y < 16; ++y)
                if (s0 + y < a.NS) ldcg_vec(a.o + (row * a.NS + s0 + y) * D + E * lane, v[y]);
        };
        if (writes) fetch(0);
        float M = fmaxf(cm, e0.x);
        for (int s = 32 + lane; s < a.NS; s += 32) M = fmaxf(M, __ldcg(ml + s).x);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        const float cf = cm == -INFINITY ? 0.f : ptx::ex2(cm - M), f0 = e0.x == -INFINITY ? 0.f : ptx::ex2(e0.x - M);
        float L = fmaf(cl, cf, e0.y * f0);
        for (int s = 32 + lane; s < a.NS; s += 32) {
            const float2 e = __ldcg(ml + s);
            L = fmaf(e.y, e.x == -INFINITY ? 0.f : ptx::ex2(e.x - M), L);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
        if (lane == 0) sm_lse[i] = M + log2f(L);
        if (!writes) continue;
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        for (int s0 = 0; s0 < a.NS; s0 += 16) {
            if (s0 > 0) fetch(s0);
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                if (s0 + y >= a.NS) break;
                const int s = s0 + y;
                float f = __shfl_sync(0xffffffffu, f0, s & 31);
                if (s >= 32) {
                    const float m = __ldcg(ml + s).x;
                    f = m == -INFINITY ? 0.f : ptx::ex2(m - M);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(v[y][e], f, acc[e]);
            }
        }
        // the cluster's states, all loads in flight together
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r < C) {
                ptx::cluster_ld_vec(ptx::cluster_addr(&join.o[0][i][E * lane], r), v[r]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) v[r][e] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float f = __shfl_sync(0xffffffffu, cf, r);  // 0 past the cluster
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(v[r][e], f, acc[e]);
        }
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) w[e / 2] = pos < 0 ? 0u : ptx::pack_bf16x2(acc[e] / L, acc[e + 1] / L);
        __nv_bfloat16* o = sa.out + row * D + E * lane;
        if constexpr (E == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(o) = w[0];
    }
    if (C > 1) ptx::cluster_arrive();  // this CTA has read the others' states
    if (SCORES) {
        __syncthreads();
        float* w = sa.weights + unit * a.S;
        for (int s = r0 + tid; s < r1; s += kAttendWarps * 32) {
            float p = 0.f;
            for (int i = 0; i < nq; ++i) p += ptx::ex2(sm_z[i * a.chunk + s - r0] - sm_lse[i]);
            w[s] += p;
        }
    }
    if (C > 1) ptx::cluster_wait();
}

// ------------------------------------------------------------------ joining the splits
constexpr int kFinishThreads = 128;
constexpr int kFinishSlots = 1024;  // slots of one key head that a CTA adds weights to

// (m*, l*) of one row over its NS splits, by a whole warp.
__device__ __forceinline__ float2 finish_ml(const float2* ml, int NS, int lane) {
    float M = -INFINITY;
    for (int s = lane; s < NS; s += 32) M = fmaxf(M, __ldcg(ml + s).x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    float L = 0.f;
    for (int s = lane; s < NS; s += 32) {  // l is 0 without a key, NaN where all its scores are
        const float2 e = __ldcg(ml + s);
        L = fmaf(e.y, e.x == -INFINITY ? 0.f : ptx::ex2(e.x - M), L);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
    return make_float2(M, L);
}

// The first B*H CTAs each write one output row; the others add the attention weights of
// kFinishSlots slots of one key head, w[slot] += sum over its G rows of 2^(z - m*) / l*, in
// the fixed order of the heads.
template <int D>
__global__ void __launch_bounds__(kFinishThreads)
    finish_kernel(const AttendArgs a, __nv_bfloat16* __restrict__ out, float* __restrict__ weights, int slot_blocks) {
    __shared__ float sm[4][D];
    extern __shared__ float sm_lse[];  // [G]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t rows = (int64_t)a.B * a.H;
    ptx::grid_dependency_wait();
    if (blockIdx.x < rows) {
        const int64_t row = blockIdx.x;
        __nv_bfloat16* orow = out + row * D;
        if (a.pos[row / a.H] < 0) {
            for (int d = tid; d < D; d += kFinishThreads) orow[d] = __float2bfloat16_rn(0.f);
            return;
        }
        const float2* ml = a.ml + row * a.NS;
        const float2 all = finish_ml(ml, a.NS, lane);
        constexpr int E = D / 32;
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int s = warp; s < a.NS; s += 4) {
            const float m = __ldcg(ml + s).x;
            if (m == -INFINITY) continue;
            const float f = ptx::ex2(m - all.x);
            float v[E];
            ldcg_vec(a.o + (row * a.NS + s) * D + E * lane, v);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(v[e], f, acc[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sm[warp][E * lane + e] = acc[e];
        __syncthreads();
        if (tid < D) orow[tid] = __float2bfloat16_rn((sm[0][tid] + sm[1][tid] + sm[2][tid] + sm[3][tid]) / all.y);
        return;
    }
    const int64_t x = blockIdx.x - rows;
    const int64_t unit = x / slot_blocks;
    const int s0 = (int)(x % slot_blocks) * kFinishSlots;
    const int64_t b = unit / a.Hkv;
    const int64_t P = a.pos[b];
    const int n = attend_slots(P, a.S, a.status, false);
    if (s0 >= n) return;
    const int64_t row0 = b * a.H + (unit % a.Hkv) * a.G;
    for (int h = warp; h < a.G; h += 4) {
        const float2 all = finish_ml(a.ml + (row0 + h) * a.NS, a.NS, lane);
        if (lane == 0) sm_lse[h] = all.x + log2f(all.y);
    }
    __syncthreads();
    const int s1 = min(s0 + kFinishSlots, n);
    for (int s = s0 + tid; s < s1; s += kFinishThreads) {
        float w = 0.f;
        for (int h = 0; h < a.G; ++h) w += ptx::ex2(a.scores[(unit * a.G + h) * a.S + s] - sm_lse[h]);
        weights[unit * a.S + s] += w;
    }
}

}  // namespace swa
