// cache_api.cu: the C ABI of the caches beside the ring (include/swa.h): key weights, the budget
// cache's seed, append and decode, and decoding behind a prefix that a whole batch shares.
// Validates arguments and launches; every check is made before anything is enqueued.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "api_internal.h"
#include "attend.cuh"
#include "cache.cuh"
#include "keyweights.cuh"
#include "prefix.cuh"
#include "swa.h"

namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return swa_internal::set_error(code, buf);
}
int success() { return swa_internal::clear_error(); }
int launched(const char* fn) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(SWA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
    return SWA_OK;
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxGroup = 1024;  // query heads to a key head

// Sizes shared by all entry points: each at least lo, the products inside 64-bit byte offsets.
int check_heads(const char* fn, int64_t B, int64_t H, int64_t Hkv, int64_t D) {
    if (B < 0 || H < 0 || Hkv < 0)
        return fail(SWA_ERR_INVALID_ARG, "%s: negative size B=%lld H=%lld Hkv=%lld", fn, (long long)B, (long long)H,
                    (long long)Hkv);
    if (D < 1) return fail(SWA_ERR_INVALID_ARG, "%s: head dim D=%lld must be >= 1", fn, (long long)D);
    if (H > 0 && (Hkv < 1 || H % Hkv != 0))
        return fail(SWA_ERR_INVALID_ARG, "%s: H=%lld is not a multiple of Hkv=%lld", fn, (long long)H, (long long)Hkv);
    if (B > INT32_MAX || H > INT32_MAX || (B > 0 && H > INT32_MAX / B))
        return fail(SWA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (H > 0 && H / Hkv > kMaxGroup)
        return fail(SWA_ERR_UNSUPPORTED, "%s: more than %lld query heads to a key head", fn, (long long)kMaxGroup);
    return SWA_OK;
}
// scale log2(e), the fp32 factor of the scores. A positive one too small for fp32 becomes the least
// that is not 0, so that a masked score, -infinity, stays that (the scores come out as 0 all the same).
int scale_log2(const char* fn, double scale, float* out) {
    if (!std::isfinite(scale)) return fail(SWA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    const double x = 1.4426950408889634 * scale;
    if (std::fabs(x) > FLT_MAX) return fail(SWA_ERR_UNSUPPORTED, "%s: scale %g is beyond fp32", fn, scale);
    *out = (float)x;
    if (scale > 0.0 && *out == 0.f) *out = FLT_TRUE_MIN;
    return SWA_OK;
}
int check_head_dim(const char* fn, int64_t D) {
    if (D != 64 && D != 128)
        return fail(SWA_ERR_UNSUPPORTED, "%s: bf16 needs D = 64 or 128 (got %lld)", fn, (long long)D);
    return SWA_OK;
}
// n operands' element strides, in[x] per dimension of size size[x] (dims of them); NULL = dense.
int read_strides(const char* fn, const int64_t* in, int n, int dims, const int64_t* size, const int64_t* dense,
                 int64_t mult, int64_t* out) {
    for (int a = 0; a < n; ++a)
        for (int x = 0; x < dims; ++x) {
            int64_t v = in ? in[dims * a + x] : dense[x];
            if (v < 0 || v > (int64_t(1) << 38))
                return fail(SWA_ERR_INVALID_ARG, "%s: stride %lld of operand %d is negative or too large", fn,
                            (long long)v, a);
            if (size[x] == 1) v = dense[x];
            if (v % mult != 0)
                return fail(SWA_ERR_MISALIGNED, "%s: bf16 strides must be multiples of 8 elements (16 bytes); operand %d "
                            "has stride %lld", fn, a, (long long)v);
            out[dims * a + x] = v;
        }
    return SWA_OK;
}

cudaLaunchConfig_t config(dim3 grid, unsigned block, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    return c;
}
// Clusters of C CTAs along x; at: the launch's one attribute.
void cluster_of(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, int C) {
    at->id = cudaLaunchAttributeClusterDimension;
    at->val.clusterDim.x = (unsigned)C;
    at->val.clusterDim.y = at->val.clusterDim.z = 1;
    cfg->attrs = at;
    cfg->numAttrs = C > 1 ? 1 : 0;
}
// A launch that may start before the kernel ahead of it on the stream has ended; the kernel
// itself waits (grid_dependency_wait).
template <typename... P, typename... A>
void launch_after(dim3 grid, unsigned block, size_t smem, cudaStream_t s, void (*kernel)(P...), A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = config(grid, block, smem, s);
    c.attrs = at;
    c.numAttrs = 1;
    cudaLaunchKernelEx(&c, kernel, args...);
}

// Let `kernel` use `bytes` of dynamic shared memory on the current device, and check that it was
// compiled with `regs` registers a thread if that is given (once a device).
int allow_smem(const void* kernel, int bytes, int regs = 0) {
    struct Done {
        int dev;
        const void* kernel;
    };
    constexpr int kMost = 256;  // more (device, kernel) pairs than that are set again each time
    static std::mutex mu;
    static Done done[kMost];
    static int n_done = 0;
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(SWA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < n_done; ++i)
        if (done[i].dev == dev && done[i].kernel == kernel) return SWA_OK;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return fail(SWA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return fail(SWA_ERR_CUDA, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
    if (regs > 0 && at.numRegs != regs)
        return fail(SWA_ERR_CUDA, "a kernel was compiled with %d registers a thread, %d expected", at.numRegs, regs);
    if (n_done < kMost) done[n_done++] = {dev, kernel};
    return SWA_OK;
}

// ------------------------------------------------------------------ key weights
template <int D>
int launch_key_weights(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const float* lse, const int64_t* lens,
                       float* weights, int64_t B, int64_t H, int64_t Hkv, int64_t T, int W, int last, float c2,
                       int* status, cudaStream_t s) {
    auto* kernel = swa::key_weights_tc_kernel<D>;
    if (int rc = allow_smem(reinterpret_cast<const void*>(kernel), swa::KwCfg<D>::kSmemBytes)) return rc;
    const int64_t tiles = (T + 127) / 128;
    // A cluster splits a key tile's query slices: while the working CTAs (the tiles that some
    // counted query sees, at most) do not give each SM one, if each keeps 4 slices or more (4 heads
    // of 1000 tokens, W 300: 7.6 us, 8.4 whole); while they do not give each SM two, if each keeps
    // 32 (4 key heads of 6000 tokens: 58 us, 90 whole; 24 slices a tile, 272 tiles: 29 us, 26 whole).
    const int64_t seen = (int64_t)W + last < T ? (int64_t)W + last : T;
    const int64_t work = B * Hkv * ((seen + 127) / 128);
    const int64_t rows = 127 + (int64_t)(W < last ? W : last);
    const int64_t slices = H / Hkv * ((rows + swa::kKwSlice - 1) / swa::kKwSlice);
    int C = 1;
    while (C < 8 && work * C < 2 * 148 && slices >= (work * C <= 74 ? 4 : 32) * C) C *= 2;
    const int64_t units = B * Hkv * tiles;
    if (units * C > INT32_MAX) C = 1;
    // Else CTAs that stay and go from tile to tile, which hides a tile's start, unless a tile is
    // long (32 heads, W 4096, 66 slices: 599 us, 580 with a CTA to each tile; W 1024, 18: 183 and 211).
    const bool stay = slices < 48 && units > 2 * 148;
    const int64_t grid = C > 1 ? units * C : stay ? 2 * 148 : units;
    cudaLaunchConfig_t cfg = config(dim3((unsigned)grid), swa::kKwThreads, swa::KwCfg<D>::kSmemBytes, s);
    cudaLaunchAttribute at[1];
    cluster_of(&cfg, at, C);
    cudaLaunchKernelEx(&cfg, kernel, tm_q, tm_k, lse, lens, weights, units, (int)H, (int)Hkv, (int)T, W,
                       last, c2, C, swa_internal::wait_limit_ns(), status);
    return SWA_OK;
}

// ------------------------------------------------------------------ decode over slots and prefix
// How one call is split. The sizes alone decide it (148 SMs assumed), so a workspace query and
// a call always agree.
struct Plan {
    int C;            // CTAs of a cluster of stream_kernel; 0: attend_kernel and finish_kernel
    int P0, pchunk0;  // prefix keys that stream_kernel reads by itself (all or none); of a CTA
    int ns, chunk;    // the streams' slots: splits; slots that a CTA takes
    int np, pchunk;   // the rest of the prefix, by prefix_kernel: splits; key tiles that a CTA takes
    bool pair;        // two row tiles a CTA
    bool early;       // stream_kernel starts beside the prefix's kernel
    int64_t NS;       // partial states a row in the workspace
    int64_t off_o, off_scores, bytes;  // workspace: (m, l), o, scores
};

void split(int64_t units, int64_t keys, int* n, int* chunk) {
    const int64_t target = 148 * 8;
    int64_t s = (target + units - 1) / units;
    int64_t c = (keys + s - 1) / s;
    c = (c + swa::kAttendStep - 1) / swa::kAttendStep * swa::kAttendStep;
    *chunk = (int)c;
    *n = (int)((keys + c - 1) / c);
}

// Key tiles that a CTA of prefix_kernel takes, of `tiles`, when `groups` CTAs take them all, on
// `sms` SMs (one CTA fits an SM): the least time, in thousandths of a tile, of rounds of their
// tiles and 3 for start and end, and for each partial state 0.08 and its part in the join of the
// `rows` query rows. *time: that, in tiles.
int prefix_chunk(int64_t groups, int tiles, int least, int64_t rows, int64_t sms, int64_t most_rounds, double* time) {
    int best = tiles;
    int64_t cost = INT64_MAX;
    for (int ns = 1; ns <= tiles && (ns == 1 || groups * ns <= most_rounds * sms); ++ns) {
        int chunk = (tiles + ns - 1) / ns;
        if (chunk < least) chunk = least;
        const int splits = (tiles + chunk - 1) / chunk;
        const int64_t c = (groups * splits + sms - 1) / sms * 1000 * (chunk + 3) + splits * (80 + rows * 80 / 1000);
        if (c < cost) {
            cost = c;
            best = chunk;
        }
    }
    *time = cost / 1000.0;
    return best;
}

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

// A prefix of at most this many bytes, taken once for each stream, is left to stream_kernel: the
// streams read it from L2, which costs less than a launch of its own and a join. Both ways were
// measured at 775 sizes (20 numbers of streams, key and query heads, D 64 and 128, 200 and 1000
// slots, 8 to 256 MB). With 8 rows, where prefix_kernel's tiles are nearly empty, they cross at 48 to
// 96 MB (with 2 rows they hardly differ, with 6 either wins); to 128 rows at 8 to 96; above, where the
// streams' query heads share what they read and prefix_kernel has twice the rows to start with, at 8
// to 192, the more slots the sooner. 8 key heads, D = 128,
// 200 slots, own and not: 8 streams, 1 head each, 64 MB 13.3 and 11.2 us, 24 MB 9.0 and 10.7; 64
// streams, 4 heads each, 48 MB 16.3 and 18.8, 96 MB 21.6 and 21.2. The choice by these three limits
// costs 4, 1 and 3 % over the faster way on average in the three ranges, 47 % (5 us) at worst.
constexpr int64_t own_prefix_bytes(int64_t rows) {
    return (rows <= swa::kAttendQueries ? 128 : rows <= 128 ? 24 : 64) << 20;
}
// Scores that a CTA of stream_kernel keeps in shared memory, in bytes.
constexpr int64_t kClusterScores = 28 << 10;

Plan plan(int64_t B, int64_t H, int64_t Hkv, int64_t S, int64_t P, int64_t D, bool scores) {
    Plan p = {};
    const int64_t G = H / Hkv, Q = swa::kAttendQueries, units = B * Hkv;
    if (G <= Q) {
        const bool own = P > 0 && (B == 1 || units * P <= own_prefix_bytes(B * G) / (4 * D));
        // The time of a call in the keys that a CTA takes meanwhile, by rates measured at the sizes
        // below and others between: rounds of resident CTAs (4 an SM for D = 128, 6 for 64; a round that is
        // not full still takes 0.55 of its time, as its CTAs share the bandwidth among fewer), each
        // its keys and 70 for its start and end, 40 for the barriers of a cluster. Of D = 128,
        // S = 1000, 192 heads: 30.3, 20.8, 27.8, 30.1 us for C = 1, 2, 4, 8; 384 heads: 38.5,
        // 48.5, 45.9, 59.4; S = 4096, 2048 heads: 680, 643, 662, 711. attend_kernel spreads over
        // all SMs but its second launch costs 290: 16 heads of S = 4096 take 16.9 us, a cluster 14.4.
        const double keys = (double)(S + (own ? P : 0)), slots = 148.0 * (D == 128 ? 4 : 6);
        double best = 1.1 * units * keys / slots + 290;
        for (int64_t C = 1; C <= 8; C *= 2) {
            const int64_t chunk = (S + 16 * C - 1) / (16 * C) * 16;
            if (scores && chunk * G * 4 > kClusterScores) continue;
            const double rounds = units * C / slots, part = rounds - std::floor(rounds);
            const double cost =
                (std::floor(rounds) + (part > 0 && part < 0.55 ? 0.55 : part)) * (keys / C + 70) + (C > 1 ? 40 : 0);
            if (cost < best) {
                best = cost;
                p.C = (int)C;
                p.chunk = (int)chunk;
                p.P0 = own ? (int)P : 0;
                p.pchunk0 = own ? (int)((P + 16 * C - 1) / (16 * C) * 16) : 0;
            }
        }
    }
    if (p.C == 0) split(units * ((G + Q - 1) / Q), S, &p.ns, &p.chunk);
    if (P > p.P0) {
        p.pair = B * G > 128;
        const int tiles = (int)((P + 127) / 128), least = p.pair ? 1 : 2;
        const int64_t groups = Hkv * (p.pair ? (B * G + 255) / 256 : 1);
        double before;
        p.pchunk = prefix_chunk(groups, tiles, least, B * H, 148, 2, &before);
        // Beside stream_kernel instead, on the SMs that its CTAs leave when all of them run at once, if
        // that is shorter (in tiles: 1.9 us, 12 MB of keys and values). 24 streams of 32 heads, 4 to a
        // key head, P 2000, S 1000 (384 CTAs): 23.9 us with 32 CTAs beside it, 31.9 with 64 before
        // it. It must not need the prefix's SMs: one that has run prefix_kernel keeps its shared-memory
        // split, with too little L1 for many loads in flight, until it is idle (the same with 64
        // CTAs beside it, which leave room for 336: 41.8 us).
        if (p.C > 0) {
            const int64_t per_sm = D == 128 ? 4 : 6, left = 148 - (units * p.C + per_sm - 1) / per_sm;
            if (left >= groups) {
                double beside;
                const int chunk = prefix_chunk(groups, tiles, least, B * H, left, 1, &beside);
                const double slots = units * S * D * 4 / 12e6, both = slots + Hkv * P * D * 4 / 12e6;
                if ((beside > both ? beside : both) < before + slots) {
                    p.pchunk = chunk;
                    p.early = true;
                }
            }
        }
        p.np = (tiles + p.pchunk - 1) / p.pchunk;
    }
    p.NS = p.ns + p.np;
    p.off_o = round256(B * H * p.NS * 8);
    p.off_scores = p.off_o + round256(B * H * p.NS * D * 4);
    p.bytes = p.off_scores + (scores && p.C == 0 ? round256(B * H * S * 4) : 0);
    return p;
}

// Sizes that plan() can take: everything below 2^31 and every byte count far inside 64 bits.
int check_decode_sizes(const char* fn, int64_t B, int64_t H, int64_t Hkv, int64_t S, int64_t P, int64_t D) {
    if (int rc = check_heads(fn, B, H, Hkv, D)) return rc;
    if (S < 1) return fail(SWA_ERR_INVALID_ARG, "%s: %lld slots, at least 1 needed", fn, (long long)S);
    if (P < 0) return fail(SWA_ERR_INVALID_ARG, "%s: negative prefix length %lld", fn, (long long)P);
    if (B == 0 || H == 0) return SWA_OK;
    if (int rc = check_head_dim(fn, D)) return rc;
    if (S > INT32_MAX / 2 || P > INT32_MAX / 2 || B * H > (int64_t(1) << 28))
        return fail(SWA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    return SWA_OK;
}

template <int D, bool PAIR>
int launch_prefix(const Plan& pl, const swa::AttendArgs& pre, cudaStream_t s) {
    using Cf = swa::PrefixCfg<D, PAIR>;
    auto* kernel = swa::prefix_kernel<D, PAIR>;
    // its register split assumes this many registers a thread at launch
    if (int rc = allow_smem(reinterpret_cast<const void*>(kernel), Cf::kSmemBytes, swa::kPPLaunchRegs)) return rc;
    CUtensorMap tm_k, tm_v;
    const int64_t P = pre.S, ks[3] = {D, pre.k_head, pre.k_row}, vs[3] = {D, pre.v_head, pre.v_row};
    if (int rc = swa_internal::tensor_map(&tm_k, pre.k, 1, pre.Hkv, P, D, ks, 128)) return rc;
    if (int rc = swa_internal::tensor_map(&tm_v, pre.v, 1, pre.Hkv, P, D, vs, 128)) return rc;
    const int64_t rows = (int64_t)pre.B * pre.G, groups = PAIR ? (rows + 255) / 256 : 1;
    const dim3 grid((unsigned)(pre.Hkv * groups), (unsigned)pl.np);
    kernel<<<grid, swa::kPrefixThreads, Cf::kSmemBytes, s>>>(tm_k, tm_v, pre, swa_internal::wait_limit_ns());
    return launched("prefix");
}

template <int D>
int launch_decode(const Plan& pl, const swa::AttendArgs& ring, const swa::AttendArgs& pre, __nv_bfloat16* out,
                  float* weights, cudaStream_t s) {
    const int Q = swa::kAttendQueries;
    const int64_t units = (int64_t)ring.B * ring.Hkv;
    const unsigned threads = swa::kAttendWarps * 32;
    if (pl.np > 0)
        if (int rc = pl.pair ? launch_prefix<D, true>(pl, pre, s) : launch_prefix<D, false>(pl, pre, s)) return rc;
    if (pl.C > 0) {
        swa::StreamArgs sa = {};
        sa.a = ring;
        sa.pk = pre.k;
        sa.pv = pre.v;
        sa.pk_head = pre.k_head;
        sa.pk_row = pre.k_row;
        sa.pv_head = pre.v_head;
        sa.pv_row = pre.v_row;
        sa.P0 = pl.P0;
        sa.pchunk = pl.pchunk0;
        sa.C = pl.C;
        sa.out = out;
        sa.weights = weights;
        cudaLaunchConfig_t cfg = config(dim3((unsigned)(units * pl.C)), threads,
                                        weights ? (size_t)pl.chunk * ring.G * 4 : 0, s);
        cudaLaunchAttribute at[2];
        unsigned n = 0;
        if (pl.C > 1) {
            at[n].id = cudaLaunchAttributeClusterDimension;
            at[n].val.clusterDim.x = (unsigned)pl.C;
            at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
            ++n;
        }
        if (pl.early) {
            at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[n].val.programmaticStreamSerializationAllowed = 1;
            ++n;
        }
        cfg.attrs = at;
        cfg.numAttrs = n;
        cudaLaunchKernelEx(&cfg, weights ? swa::stream_kernel<D, true> : swa::stream_kernel<D, false>, sa);
        return SWA_OK;
    }
    const dim3 grid((unsigned)(units * ((ring.G + Q - 1) / Q)), (unsigned)pl.ns);
    if (weights) swa::attend_kernel<D, true><<<grid, threads, 0, s>>>(ring);
    else swa::attend_kernel<D, false><<<grid, threads, 0, s>>>(ring);
    const int slot_blocks = weights ? (ring.S + swa::kFinishSlots - 1) / swa::kFinishSlots : 0;
    const int64_t blocks = (int64_t)ring.B * ring.H + units * slot_blocks;
    launch_after(dim3((unsigned)blocks), swa::kFinishThreads, (size_t)ring.G * 4, s, swa::finish_kernel<D>, ring, out,
                 weights, slot_blocks);
    return SWA_OK;
}

int decode(const char* fn, const void* q, const void* k, const void* v, const int64_t* pos, const void* kp, const void* vp,
           float* weights, bool scores, void* out, void* workspace, int64_t workspace_bytes, int64_t B, int64_t H,
           int64_t Hkv, int64_t S, int64_t P, int64_t D, double scale, const int64_t* strides, void* stream) {
    if (int rc = check_decode_sizes(fn, B, H, Hkv, S, P, D)) return rc;
    float c2;
    if (int rc = scale_log2(fn, scale, &c2)) return rc;
    if (B == 0 || H == 0) return success();
    if (!(scale > 0.0)) return fail(SWA_ERR_UNSUPPORTED, "%s: scale must be > 0 (got %g)", fn, scale);
    if (!q || !k || !v || !pos || !out || (scores && !weights) || (P > 0 && (!kp || !vp)))
        return fail(SWA_ERR_INVALID_ARG, "%s: null pointer", fn);
    const Plan pl = plan(B, H, Hkv, S, P, D, scores);
    if (pl.bytes > 0 && !workspace) return fail(SWA_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (workspace_bytes < pl.bytes)
        return fail(SWA_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", fn, (long long)workspace_bytes,
                    (long long)pl.bytes);
    const void* p16[] = {q, k, v, out, P > 0 ? kp : nullptr, P > 0 ? vp : nullptr};
    for (const void* x : p16)
        if (!aligned(x, 16)) return fail(SWA_ERR_MISALIGNED, "%s: tensors must be 16-byte aligned", fn);
    if (!aligned(workspace, 256) || !aligned(pos, 8) || (scores && !aligned(weights, 4)))
        return fail(SWA_ERR_MISALIGNED, "%s: workspace must be 256-byte, pos 8-byte and weights 4-byte aligned", fn);
    int64_t st[4] = {0, 0, 0, 0};
    if (P > 0) {
        const int64_t size[2] = {Hkv, P}, dense[2] = {P * D, D};
        if (int rc = read_strides(fn, strides, 2, 2, size, dense, 8, st)) return rc;
    }
    const int64_t G = H / Hkv;
    const int64_t blocks = B * H + (scores ? B * Hkv * ((S + swa::kFinishSlots - 1) / swa::kFinishSlots) : 0);
    if (blocks > INT32_MAX || B * Hkv > INT32_MAX / 8 || pl.ns > 65535) return fail(SWA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    int *status, num_sms;
    if (int rc = swa_internal::device_info(&status, &num_sms)) return rc;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    swa::AttendArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.pos = pos;
    a.ml = reinterpret_cast<float2*>(ws);
    a.o = reinterpret_cast<float*>(ws + pl.off_o);
    a.scores = scores ? reinterpret_cast<float*>(ws + pl.off_scores) : nullptr;
    a.k_head = a.v_head = S * D;
    a.k_row = a.v_row = D;
    a.B = (int)B;
    a.H = (int)H;
    a.Hkv = (int)Hkv;
    a.G = (int)G;
    a.S = (int)S;
    a.chunk = pl.chunk;
    a.split0 = pl.np;  // the prefix's partial states come first
    a.NS = (int)pl.NS;
    a.scale_log2 = c2;
    a.status = status;
    swa::AttendArgs pre = a;
    pre.k = static_cast<const __nv_bfloat16*>(kp);
    pre.v = static_cast<const __nv_bfloat16*>(vp);
    pre.k_head = st[0];
    pre.k_row = st[1];
    pre.v_head = st[2];
    pre.v_row = st[3];
    pre.S = (int)P;
    pre.chunk = pl.pchunk;
    pre.split0 = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto* ob = static_cast<__nv_bfloat16*>(out);
    float* w = scores ? weights : nullptr;
    if (int rc = D == 128 ? launch_decode<128>(pl, a, pre, ob, w, s) : launch_decode<64>(pl, a, pre, ob, w, s)) return rc;
    if (int rc = launched(fn)) return rc;
    return success();
}

int64_t decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t S, int64_t P, int64_t D, bool scores) {
    if (check_decode_sizes("workspace size", B, H, Hkv, S, P, D)) return -1;
    if (B == 0 || H == 0) return 0;
    return plan(B, H, Hkv, S, P, D, scores).bytes;
}

}  // namespace

extern "C" {

int swa_key_weights(const void* q, const void* k, const float* lse, const int64_t* lens, float* weights, int64_t B,
                    int64_t H, int64_t Hkv, int64_t T, int64_t D, int64_t W, int64_t last, double scale,
                    const int64_t* strides, int dtype, void* stream) {
    const char* fn = "swa_key_weights";
    if (dtype != SWA_F32 && dtype != SWA_BF16)
        return fail(SWA_ERR_INVALID_ARG, "%s: dtype %d is neither SWA_F32 nor SWA_BF16", fn, dtype);
    if (int rc = check_heads(fn, B, H, Hkv, D)) return rc;
    if (T < 0) return fail(SWA_ERR_INVALID_ARG, "%s: negative size T=%lld", fn, (long long)T);
    if (W < 1) return fail(SWA_ERR_INVALID_ARG, "%s: window W=%lld must be >= 1", fn, (long long)W);
    if (last < 1) return fail(SWA_ERR_INVALID_ARG, "%s: last=%lld must be >= 1", fn, (long long)last);
    float c2;
    if (int rc = scale_log2(fn, scale, &c2)) return rc;
    if (B == 0 || Hkv == 0 || T == 0) return success();
    if (!weights || (H > 0 && (!q || !k || !lse))) return fail(SWA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (Hkv > INT32_MAX || B > INT32_MAX / Hkv) return fail(SWA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (dtype == SWA_BF16) {
        if (int rc = check_head_dim(fn, D)) return rc;
    } else if (D > 4096) {
        return fail(SWA_ERR_UNSUPPORTED, "%s: fp32 supports D <= 4096", fn);
    }
    const int64_t n_kt = (T + swa::kKwTile - 1) / swa::kKwTile;
    if (T > (int64_t(1) << 29) || B * Hkv > INT32_MAX / n_kt) return fail(SWA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    const size_t al = dtype == SWA_BF16 ? 16 : 4;
    if (!aligned(q, al) || !aligned(k, al))
        return fail(SWA_ERR_MISALIGNED, "%s: q and k must be %d-byte aligned", fn, (int)al);
    if (!aligned(lse, 4) || !aligned(weights, 4) || !aligned(lens, 8))
        return fail(SWA_ERR_MISALIGNED, "%s: lse and weights must be 4-byte and lens 8-byte aligned", fn);
    int64_t qs[3], ks[3];
    {
        const int64_t size[3] = {B, H, T}, dense[3] = {H * T * D, T * D, D};
        if (int rc = read_strides(fn, strides, 1, 3, size, dense, dtype == SWA_BF16 ? 8 : 1, qs)) return rc;
        const int64_t ksize[3] = {B, Hkv, T}, kdense[3] = {Hkv * T * D, T * D, D};
        if (int rc = read_strides(fn, strides ? strides + 3 : nullptr, 1, 3, ksize, kdense, dtype == SWA_BF16 ? 8 : 1, ks))
            return rc;
    }
    const int Wi = (int)(W < T ? W : T), Li = (int)(last < T ? last : T);
    int *status, num_sms;
    if (int rc = swa_internal::device_info(&status, &num_sms)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SWA_BF16 && H > 0) {
        CUtensorMap tm_q, tm_k;
        if (int rc = swa_internal::tensor_map(&tm_q, q, B, H, T, D, qs, swa::kKwSlice)) return rc;
        if (int rc = swa_internal::tensor_map(&tm_k, k, B, Hkv, T, D, ks, 128)) return rc;
        if (int rc = D == 128 ? launch_key_weights<128>(tm_q, tm_k, lse, lens, weights, B, H, Hkv, T, Wi, Li, c2, status, s)
                              : launch_key_weights<64>(tm_q, tm_k, lse, lens, weights, B, H, Hkv, T, Wi, Li, c2, status, s))
            return rc;
    } else {
        // (also for no query heads of either type: every sum is 0 and q, k, lse are not read)
        // a cluster splits the query tiles while the CTAs do not fill the SMs twice
        const int64_t units = B * Hkv * n_kt, tiles = H / Hkv * ((swa::kKwTile + (Wi < Li ? Wi : Li) + 62) / swa::kKwTile);
        int C = 1;
        while (C < 8 && units * C < 2 * 148 && tiles >= 2 * C) C *= 2;
        cudaLaunchConfig_t cfg = config(dim3((unsigned)(units * C)), swa::kKwSimtThreads, 0, s);
        cudaLaunchAttribute at[1];
        cluster_of(&cfg, at, C);
        cudaLaunchKernelEx(&cfg, swa::key_weights_simt_kernel, static_cast<const float*>(q), static_cast<const float*>(k),
                           lse, lens, weights, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], (int)H, (int)Hkv, (int)T, (int)D,
                           Wi, Li, (float)scale, (int)n_kt, C, status);
    }
    if (int rc = launched(fn)) return rc;
    return success();
}

int swa_cache_seed(const void* k, const void* v, const float* weights, const int64_t* lens, void* kcache, void* vcache,
                   float* wcache, int64_t* pcache, int64_t B, int64_t Hkv, int64_t T, int64_t D, int64_t S, int64_t recent,
                   const int64_t* strides, void* stream) {
    const char* fn = "swa_cache_seed";
    if (int rc = check_heads(fn, B, Hkv, Hkv, D)) return rc;
    if (T < 0) return fail(SWA_ERR_INVALID_ARG, "%s: negative size T=%lld", fn, (long long)T);
    if (S < 1) return fail(SWA_ERR_INVALID_ARG, "%s: %lld slots, at least 1 needed", fn, (long long)S);
    if (recent < 0 || recent >= S)
        return fail(SWA_ERR_INVALID_ARG, "%s: recent=%lld must be in [0, %lld)", fn, (long long)recent, (long long)S);
    if (B == 0 || Hkv == 0 || T == 0) return success();
    if (!k || !v || !weights || !kcache || !vcache || !wcache || !pcache)
        return fail(SWA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (int rc = check_head_dim(fn, D)) return rc;
    if (T > INT32_MAX / 2 || S > INT32_MAX / 2 || B * Hkv > INT32_MAX / 8)
        return fail(SWA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kcache, 16) || !aligned(vcache, 16))
        return fail(SWA_ERR_MISALIGNED, "%s: key and value tensors must be 16-byte aligned", fn);
    if (!aligned(weights, 4) || !aligned(wcache, 4) || !aligned(pcache, 8) || !aligned(lens, 8))
        return fail(SWA_ERR_MISALIGNED, "%s: weights must be 4-byte, positions and lens 8-byte aligned", fn);
    int64_t st[6];
    const int64_t size[3] = {B, Hkv, T}, dense[3] = {Hkv * T * D, T * D, D};
    if (int rc = read_strides(fn, strides, 2, 3, size, dense, 8, st)) return rc;
    int *status, num_sms;
    if (int rc = swa_internal::device_info(&status, &num_sms)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // A cluster while the heads alone do not fill the SMs, each CTA keeping a step's worth of
    // positions.
    int C = 1;
    while (C < 8 && B * Hkv * C < 148 && T >= 2 * C * swa::kSeedThreads) C *= 2;
    cudaLaunchConfig_t cfg = config(dim3((unsigned)(B * Hkv * C)), swa::kSeedThreads, 0, s);
    cudaLaunchAttribute at[1];
    cluster_of(&cfg, at, C);
    cudaLaunchKernelEx(&cfg, swa::cache_seed_kernel, static_cast<const __nv_bfloat16*>(k),
                       static_cast<const __nv_bfloat16*>(v), weights, lens, static_cast<uint4*>(kcache),
                       static_cast<uint4*>(vcache), wcache, pcache, st[0], st[1], st[2], st[3], st[4], st[5], (int)Hkv,
                       (int)T, (int)S, (int)recent, (int)(D / 8), C, status);
    if (int rc = launched(fn)) return rc;
    return success();
}

int swa_cache_append(const void* k, const void* v, void* kcache, void* vcache, float* wcache, int64_t* pcache,
                     const int64_t* pos, int64_t* slots, int64_t B, int64_t Hkv, int64_t D, int64_t S, int64_t recent,
                     void* stream) {
    const char* fn = "swa_cache_append";
    if (int rc = check_heads(fn, B, Hkv, Hkv, D)) return rc;
    if (S < 1) return fail(SWA_ERR_INVALID_ARG, "%s: %lld slots, at least 1 needed", fn, (long long)S);
    if (recent < 0 || recent >= S)
        return fail(SWA_ERR_INVALID_ARG, "%s: recent=%lld must be in [0, %lld)", fn, (long long)recent, (long long)S);
    if (B == 0 || Hkv == 0) return success();
    if (!k || !v || !kcache || !vcache || !wcache || !pcache || !pos || !slots)
        return fail(SWA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (int rc = check_head_dim(fn, D)) return rc;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kcache, 16) || !aligned(vcache, 16))
        return fail(SWA_ERR_MISALIGNED, "%s: key and value tensors must be 16-byte aligned", fn);
    if (!aligned(wcache, 4) || !aligned(pcache, 8) || !aligned(pos, 8) || !aligned(slots, 8))
        return fail(SWA_ERR_MISALIGNED, "%s: weights must be 4-byte, positions and slots 8-byte aligned", fn);
    if (S > INT32_MAX / 2) return fail(SWA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    int *status, num_sms;
    if (int rc = swa_internal::device_info(&status, &num_sms)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    swa::cache_append_kernel<<<(unsigned)(B * Hkv), swa::kAppendThreads, 0, s>>>(
        static_cast<const uint4*>(k), static_cast<const uint4*>(v), static_cast<uint4*>(kcache),
        static_cast<uint4*>(vcache), wcache, pcache, pos, slots, (int)Hkv, (int)S, (int)recent, (int)(D / 8), status);
    if (int rc = launched(fn)) return rc;
    return success();
}

int64_t swa_cache_decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t S, int64_t P, int64_t D) {
    return decode_workspace_bytes(B, H, Hkv, S, P, D, true);
}

int swa_cache_decode(const void* q, const void* kcache, const void* vcache, float* wcache, const int64_t* pos,
                     const void* kprefix, const void* vprefix, void* out, void* workspace, int64_t workspace_bytes,
                     int64_t B, int64_t H, int64_t Hkv, int64_t S, int64_t P, int64_t D, double scale,
                     const int64_t* strides, void* stream) {
    return decode("swa_cache_decode", q, kcache, vcache, pos, kprefix, vprefix, wcache, true, out, workspace,
                  workspace_bytes, B, H, Hkv, S, P, D, scale, strides, stream);
}

int64_t swa_prefix_decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t W, int64_t P, int64_t D) {
    return decode_workspace_bytes(B, H, Hkv, W, P, D, false);
}

int swa_prefix_decode(const void* q, const void* kprefix, const void* vprefix, const void* kring, const void* vring,
                      const int64_t* pos, void* out, void* workspace, int64_t workspace_bytes, int64_t B, int64_t H,
                      int64_t Hkv, int64_t W, int64_t P, int64_t D, double scale, const int64_t* strides, void* stream) {
    return decode("swa_prefix_decode", q, kring, vring, pos, kprefix, vprefix, nullptr, false, out, workspace,
                  workspace_bytes, B, H, Hkv, W, P, D, scale, strides, stream);
}

}  // extern "C"
