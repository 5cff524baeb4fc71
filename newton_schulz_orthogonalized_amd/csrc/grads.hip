// Global gradient norm and clipping over lists of tensors (gfx950): the C
// entry points and their kernels.
//
//   s = sum over tensors and elements of g^2      (float64, fixed order)
//   norm = sqrt(s),  c = min(1, max_norm / (norm + eps)),  out = c g
//
// A list travels in the kernels' arguments (no descriptor table in device
// memory, so a call can be captured into a graph), SQ_SEGS or CLIP_SEGS
// tensors a launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "../../include/muon_mi355x.h"
#include "capi_common.hpp"
#include "common.hpp"

using namespace mu;

namespace {

constexpr int NTHR = 256;
constexpr int GRAD_CHUNK = 8192;    // elements a workgroup takes at a time
constexpr int SQ_WGS = 1024;        // workgroups (and float64 partial sums) of one launch
constexpr int CLIP_WGS = 512;

// A tensor's elements; chunk c of the launch belongs to the last segment with c0 <= c.
struct SqSeg {
    const void* p;
    int64_t n;
    int32_t c0;
    int32_t dtype;
};
constexpr int SQ_SEGS = 160;
struct SqArgs {
    SqSeg seg[SQ_SEGS];
    double* partials;   // gridDim.x of them
    int nseg;
    int chunks;
};
static_assert(sizeof(SqArgs) <= 4096, "kernel arguments");

// How norm and c leave the sums.
struct NormOut {
    const double* partials;
    int n;
    float max_norm, eps;
    float* norm;
    float* scale;
};

struct ClipSeg {
    const void* p;
    void* out;
    int64_t n;
    int32_t c0;
    int16_t dtype, out_dtype;
};
constexpr int CLIP_SEGS = 120;
struct ClipArgs {
    ClipSeg seg[CLIP_SEGS];
    NormOut no;
    int nseg;
    int chunks;
};
static_assert(sizeof(ClipArgs) <= 4096, "kernel arguments");

__device__ __forceinline__ double block_sum(double v, double* red) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const double s = ((red[0] + red[1]) + red[2]) + red[3];
    __syncthreads();
    return s;
}

// Sum of squares of a chunk (elements i0 .. of a tensor of n). Squares of
// float32 values are exact in float64, whose additions hide behind the loads.
// Bound by memory: every load of a chunk is in flight before the first square,
// and non-temporal (Llama-1B-shaped set, 2.68 GB of bfloat16: 529 us with loads
// as they come, 440 with all of a chunk's first, 393 non-temporal (NT), 6.8 TB/s;
// one run of chunks for each XCD 414-418, 2048 workgroups 432).
// (Vectors at element alignment here and below: gfx950 takes global vector
// accesses at any address, so tensors that start anywhere in an allocation need
// no other path.)
template <bool NT, typename T>
__device__ __forceinline__ double sumsq_chunk(const void* base, int64_t i0, int64_t n, int tid) {
    const MU_GLOBAL T* p = (const MU_GLOBAL T*)base + i0;
    constexpr int EPV = 16 / (int)sizeof(T), STEPS = GRAD_CHUNK / (NTHR * EPV);
    typedef T V __attribute__((ext_vector_type(EPV)));
    typedef V VU __attribute__((aligned(sizeof(T))));
    double s = 0.0;
    const int64_t left = n - i0;
    if (left >= GRAD_CHUNK) {
        V v[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const MU_GLOBAL VU* q = (const MU_GLOBAL VU*)(p + (k * NTHR + tid) * EPV);
            if constexpr (NT) v[k] = __builtin_nontemporal_load(q);
            else v[k] = *q;
        }
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const double x = (double)(float)v[k][e];
                s = fma(x, x, s);
            }
        return s;
    }
    for (int i = tid * EPV; i < (int)left; i += NTHR * EPV) {
        V v;
        if (i + EPV <= left) v = *(const MU_GLOBAL VU*)(p + i);
        else
#pragma unroll
            for (int e = 0; e < EPV; ++e) v[e] = i + e < left ? p[i + e] : (T)0.f;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const double x = (double)(float)v[e];
            s = fma(x, x, s);
        }
    }
    return s;
}

// The segment of chunk c: the last one that starts at or before it, found by
// all lanes of a wave at once.
template <typename Seg>
__device__ __forceinline__ int seg_of(const Seg* seg, int n, int c) {
    int before = 0;
    for (int j = 0; j < n; j += 64) {
        const int k = j + (int)(threadIdx.x & 63);
        before += __popcll(__ballot(k < n && seg[min(k, n - 1)].c0 <= c));
    }
    return __builtin_amdgcn_readfirstlane(before - 1);
}

template <bool NT>
__device__ __forceinline__ double sumsq_of(const SqSeg& S, int c, int tid) {
    const int64_t i0 = (int64_t)(c - S.c0) * GRAD_CHUNK;
    return S.dtype == DT_BF16 ? sumsq_chunk<NT, bf16>(S.p, i0, S.n, tid) : sumsq_chunk<NT, float>(S.p, i0, S.n, tid);
}

template <bool NT>
__global__ __launch_bounds__(NTHR) void k_sumsq(SqArgs A) {
    __shared__ double red[4];
    double s = 0.0;
    int i = (int)blockIdx.x < A.chunks ? seg_of(A.seg, A.nseg, blockIdx.x) : 0;
    for (int c = blockIdx.x; c < A.chunks; c += gridDim.x) {
        while (i + 1 < A.nseg && A.seg[i + 1].c0 <= c) ++i;
        s += sumsq_of<NT>(A.seg[i], c, threadIdx.x);
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0) gp(A.partials)[blockIdx.x] = s;
}

// norm and c from the sum of squares; written where `writes`. Returns c.
__device__ __forceinline__ float norm_out(const NormOut& N, double s, bool writes) {
    const double norm = sqrt(s);
    const double r = (double)N.max_norm / (norm + (double)N.eps);
    // 0 / 0 (both bounds 0 and no gradient) and inf / inf (no bound and an infinite
    // norm) clip nothing; a NaN norm stays NaN
    const float c = isnan(norm) ? (float)norm : (r < 1.0 ? (float)r : 1.f);
    if (writes) {
        if (N.norm) *gp(N.norm) = (float)norm;
        if (N.scale) *gp(N.scale) = c;
    }
    return c;
}

// The sum of the partials in a fixed order, by every thread of a workgroup.
__device__ __forceinline__ double sum_partials(const NormOut& N, double* red) {
    double s = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < N.n; i += NTHR) s += gp(N.partials)[i];
    return block_sum(s, red);
}

__global__ __launch_bounds__(NTHR) void k_norm_final(NormOut N) {
    __shared__ double red[4];
    norm_out(N, sum_partials(N, red), threadIdx.x == 0);
}

// A chunk times c (float32, as the product before it is rounded to the output's
// type), all loads before the first store. Bound by memory: four layers
// and the embedding of the Llama-1B-shaped set, float32 into bfloat16, norm and
// scaling together (2.7 GB): 478 us, 461 with the loads first, 429 with
// non-temporal loads and stores, 417 with CLIP_WGS = 512 rather than 1024
// workgroups; going through the chunks backwards, last read first, gained nothing.
template <bool NT, typename TI, typename TO>
__device__ __forceinline__ void clip_chunk(const void* base, void* out, int64_t i0, int64_t n, float c, int tid) {
    const MU_GLOBAL TI* p = (const MU_GLOBAL TI*)base + i0;
    MU_GLOBAL TO* o = (MU_GLOBAL TO*)out + i0;
    constexpr int EPV = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4, STEPS = GRAD_CHUNK / (NTHR * EPV);
    typedef TI VI __attribute__((ext_vector_type(EPV)));
    typedef TO VO __attribute__((ext_vector_type(EPV)));
    typedef VI VIU __attribute__((aligned(sizeof(TI))));
    typedef VO VOU __attribute__((aligned(sizeof(TO))));
    const int64_t left = n - i0;
    if (left >= GRAD_CHUNK) {
        VI v[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const MU_GLOBAL VIU* q = (const MU_GLOBAL VIU*)(p + (k * NTHR + tid) * EPV);
            if constexpr (NT) v[k] = __builtin_nontemporal_load(q);
            else v[k] = *q;
        }
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            VO r;
#pragma unroll
            for (int e = 0; e < EPV; ++e) r[e] = (TO)(c * (float)v[k][e]);
            MU_GLOBAL VOU* q = (MU_GLOBAL VOU*)(o + (k * NTHR + tid) * EPV);
            if constexpr (NT) __builtin_nontemporal_store(r, q);
            else *q = r;
        }
        return;
    }
    for (int i = tid * EPV; i < (int)left; i += NTHR * EPV) {
        if (i + EPV <= left) {
            const VI v = *(const MU_GLOBAL VIU*)(p + i);
            VO r;
#pragma unroll
            for (int e = 0; e < EPV; ++e) r[e] = (TO)(c * (float)v[e]);
            *(MU_GLOBAL VOU*)(o + i) = r;
        } else {
            for (int j = i; j < (int)left; ++j) o[j] = (TO)(c * (float)p[j]);
        }
    }
}

template <bool NT>
__device__ __forceinline__ void clip_of(const ClipSeg& S, int q, float c, int tid) {
    if (c == 1.f && S.p == S.out) return;   // in place and nothing to clip
    const int64_t i0 = (int64_t)(q - S.c0) * GRAD_CHUNK;
    if (S.dtype == DT_BF16) {
        if (S.out_dtype == DT_BF16) clip_chunk<NT, bf16, bf16>(S.p, S.out, i0, S.n, c, tid);
        else clip_chunk<NT, bf16, float>(S.p, S.out, i0, S.n, c, tid);
    } else {
        if (S.out_dtype == DT_BF16) clip_chunk<NT, float, bf16>(S.p, S.out, i0, S.n, c, tid);
        else clip_chunk<NT, float, float>(S.p, S.out, i0, S.n, c, tid);
    }
}

template <bool NT>
__global__ __launch_bounds__(NTHR) void k_clip(ClipArgs A) {
    __shared__ double red[4];
    int i = (int)blockIdx.x < A.chunks ? seg_of(A.seg, A.nseg, blockIdx.x) : 0;
    const float c = norm_out(A.no, sum_partials(A.no, red), blockIdx.x == 0 && threadIdx.x == 0);
    for (int q = blockIdx.x; q < A.chunks; q += gridDim.x) {
        while (i + 1 < A.nseg && A.seg[i + 1].c0 <= q) ++i;
        const ClipSeg S = A.seg[i];
        clip_of<NT>(S, q, c, threadIdx.x);
    }
}

// A few chunks in one launch of one workgroup: its four quarters take a chunk
// each at a time, and for clipping read theirs again from the caches. Whole
// calls on one float32 tensor, in one launch and in two: norm of 16 chunks 11.8
// and 14.2 us, of 32 11.8 and 14.3, of 64 26.2 and 14.3; clipping of 12 chunks
// 12.9 and 15.8, of 16 17.3 and 15.7, of 32 32.1 and 15.8.
constexpr int FEW_NORM = 32, FEW_CLIP = 12, FEW_THR = 4 * NTHR;
static_assert(FEW_NORM <= CLIP_SEGS && FEW_CLIP <= CLIP_SEGS, "one launch takes the segments of so few chunks");
template <bool CLIP>
__global__ __launch_bounds__(FEW_THR) void k_few(ClipArgs A) {
    __shared__ double red[FEW_THR / 64];
    const int tid = threadIdx.x % NTHR, quarter = __builtin_amdgcn_readfirstlane(threadIdx.x / NTHR);
    double s = 0.0;
    for (int q = quarter; q < A.chunks; q += 4) {
        const ClipSeg& S = A.seg[seg_of(A.seg, A.nseg, q)];
        s += sumsq_of<false>(SqSeg{S.p, S.n, S.c0, S.dtype}, q, tid);
    }
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < FEW_THR / 64; ++w) s += red[w];
    const float c = norm_out(A.no, s, threadIdx.x == 0);
    if constexpr (CLIP) {
        for (int q = quarter; q < A.chunks; q += 4) {
            const ClipSeg S = A.seg[seg_of(A.seg, A.nseg, q)];
            clip_of<false>(S, q, c, tid);
        }
    }
}

// Memory of a call up to which it leaves what it touches in the caches (256 MB
// the last level), as the step reads it next. Gradients just written, clipped,
// then read once more, non-temporal and not: 48 MB of float32 into bfloat16 64
// and 55 us, in place 70 and 60; 160 MB (240 with the outputs) 189 and 175, in
// place 211 and 191; 224 MB in place 310 and 274, into bfloat16 (336) 274 and 281;
// 320 MB in place 452 and 489. Their norm and a reader: 32 MB 48 and 37 us, 96 MB
// 107 and 94, 224 MB 238 and 207 (the norm alone, read again and again, 15.8 and
// 15.7, 17.1 and 18.7, 36.7 and 37.7; 320 MB 51 and 56).
constexpr double CACHED = 256 << 20;

size_t es_of(int dt) { return dt == MU_BF16 ? 2 : 4; }

int check_list(const mu_grad* gs, int32_t n, bool with_out, const float* norm_out, const float* scale_out) {
    if (n < 0) return fail(MU_ERR_INVALID_ARG, "n must be >= 0");
    if (n > 0 && !gs) return fail(MU_ERR_INVALID_ARG, "gradient list is null");
    std::vector<Range> ranges;
    for (const float* p : {norm_out, scale_out})
        if (p) ranges.push_back({(uintptr_t)p, (uintptr_t)p + 4, -1});
    for (int i = 0; i < n; ++i) {
        const mu_grad& g = gs[i];
        if (g.dtype != MU_F32 && g.dtype != MU_BF16) return fail(MU_ERR_DTYPE, "gradient %d: unknown dtype %d", i, g.dtype);
        if (g.numel < 0 || g.numel > ((int64_t)1 << 42)) return fail(MU_ERR_INVALID_ARG, "gradient %d: bad numel", i);
        if (g.numel > 0 && !g.grad) return fail(MU_ERR_INVALID_ARG, "gradient %d: null buffer", i);
        if (!aligned(g.grad, es_of(g.dtype))) return fail(MU_ERR_LAYOUT, "gradient %d: misaligned buffer", i);
        if (!with_out) continue;
        if (g.out_dtype != MU_F32 && g.out_dtype != MU_BF16)
            return fail(MU_ERR_DTYPE, "gradient %d: unknown output dtype %d", i, g.out_dtype);
        if (g.numel > 0 && !g.out) return fail(MU_ERR_INVALID_ARG, "gradient %d: null output", i);
        if (!aligned(g.out, es_of(g.out_dtype))) return fail(MU_ERR_LAYOUT, "gradient %d: misaligned output", i);
        if (g.numel > 0) {
            ranges.push_back({(uintptr_t)g.grad, (uintptr_t)g.grad + (size_t)g.numel * es_of(g.dtype), i});
            if (g.out != g.grad || g.out_dtype != g.dtype)
                ranges.push_back({(uintptr_t)g.out, (uintptr_t)g.out + (size_t)g.numel * es_of(g.out_dtype), i});
        }
    }
    if (ranges_overlap(ranges)) return fail(MU_ERR_LAYOUT, "buffers of the gradient list overlap");
    return MU_OK;
}

int64_t chunks_of(int64_t numel) { return (numel + GRAD_CHUNK - 1) / GRAD_CHUNK; }

// The list's tensors that hold elements, in launches of at most `segs` of them
// and 2^30 chunks in all (a tensor of 2^42 elements has 2^29).
struct Batch {
    std::vector<int> items;
    int64_t chunks = 0;
};
void batches(const mu_grad* gs, int32_t n, int segs, std::vector<Batch>& out) {
    out.clear();
    for (int i = 0; i < n; ++i) {
        if (gs[i].numel == 0) continue;
        const int64_t c = chunks_of(gs[i].numel);
        if (out.empty() || (int)out.back().items.size() == segs || out.back().chunks + c > (1 << 30)) out.emplace_back();
        out.back().items.push_back(i);
        out.back().chunks += c;
    }
}

// Workgroups of a launch over so many chunks: a multiple of 8, so that every XCD has some.
int wgs_of(int64_t chunks, int most) { return (int)std::min<int64_t>((chunks + 7) / 8 * 8, most); }
size_t partials_of(const std::vector<Batch>& b) {
    size_t p = 0;
    for (auto& x : b) p += (size_t)wgs_of(x.chunks, SQ_WGS);
    return p;
}

int norm_and_clip(const mu_grad* gs, int32_t n, float max_norm, float eps, float* norm_out, float* scale_out, bool clip,
                  void* ws, size_t ws_bytes, hipStream_t s) {
    int rc = check_list(gs, n, clip, norm_out, scale_out);
    if (rc) return rc;
    if (!(max_norm >= 0.f)) return fail(MU_ERR_INVALID_ARG, "max_norm must be >= 0");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(MU_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!clip && !norm_out && !scale_out) return fail(MU_ERR_INVALID_ARG, "norm_out and scale_out are both null");
    if (!aligned(norm_out, 4) || !aligned(scale_out, 4)) return fail(MU_ERR_LAYOUT, "misaligned norm_out or scale_out");
    std::vector<Batch> bs;
    batches(gs, n, SQ_SEGS, bs);
    const size_t np = partials_of(bs), need = align_up(np * sizeof(double));
    if (np) {
        if (!ws) return fail(MU_ERR_WORKSPACE, "workspace is null (need %zu bytes)", need);
        if (!aligned(ws, ALIGN)) return fail(MU_ERR_WORKSPACE, "workspace must be 256-byte aligned");
        if (ws_bytes < need) return fail(MU_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    }
    auto clip_args = [&](const Batch& b, ClipArgs& a) {
        double bytes = 0;
        int64_t c = 0;
        a.nseg = (int)b.items.size();
        for (int k = 0; k < a.nseg; ++k) {
            const mu_grad& g = gs[b.items[k]];
            a.seg[k] = ClipSeg{g.grad, g.out, g.numel, (int32_t)c, (int16_t)g.dtype, (int16_t)g.out_dtype};
            c += chunks_of(g.numel);
            bytes += (double)g.numel * (es_of(g.dtype) + (clip ? es_of(g.out_dtype) : 0));
        }
        a.chunks = (int)c;
        return bytes;
    };
    if (bs.size() == 1 && bs[0].chunks <= (clip ? FEW_CLIP : FEW_NORM)) {
        ClipArgs a;
        const double bytes = clip_args(bs[0], a);
        a.no = NormOut{nullptr, 0, max_norm, eps, norm_out, scale_out};
        return timed_launch(clip ? MU_K_CLIP : MU_K_GRADNORM, 0.0, bytes, s, [&] {
            if (clip) hipLaunchKernelGGL(k_few<true>, dim3(1), dim3(FEW_THR), 0, s, a);
            else hipLaunchKernelGGL(k_few<false>, dim3(1), dim3(FEW_THR), 0, s, a);
            return hipGetLastError();
        }, "gradient norm launch");
    }
    double memory = 0;
    for (int i = 0; i < n; ++i)
        memory += (double)gs[i].numel * (es_of(gs[i].dtype) + (clip && gs[i].out != gs[i].grad ? es_of(gs[i].out_dtype) : 0));
    const bool nt = memory > CACHED;
    double* part = (double*)ws;
    for (auto& b : bs) {
        SqArgs a;
        double bytes = 0;
        int64_t c = 0;
        a.nseg = (int)b.items.size();
        for (int k = 0; k < a.nseg; ++k) {
            const mu_grad& g = gs[b.items[k]];
            a.seg[k] = SqSeg{g.grad, g.numel, (int32_t)c, g.dtype};
            c += chunks_of(g.numel);
            bytes += (double)g.numel * es_of(g.dtype);
        }
        a.chunks = (int)c;
        a.partials = part;
        const int grid = wgs_of(c, SQ_WGS);
        part += grid;
        rc = timed_launch(MU_K_GRADNORM, 0.0, bytes, s, [&] {
            if (nt) hipLaunchKernelGGL(k_sumsq<true>, dim3(grid), dim3(NTHR), 0, s, a);
            else hipLaunchKernelGGL(k_sumsq<false>, dim3(grid), dim3(NTHR), 0, s, a);
            return hipGetLastError();
        }, "gradient norm launch");
        if (rc) return rc;
    }
    NormOut no{(const double*)ws, (int)np, max_norm, eps, norm_out, scale_out};
    if (!clip || bs.empty()) {
        if (!norm_out && !scale_out) return MU_OK;
        return timed_launch(MU_K_GRADNORM, 0.0, 8.0 * (double)np, s, [&] {
            hipLaunchKernelGGL(k_norm_final, dim3(1), dim3(NTHR), 0, s, no);
            return hipGetLastError();
        }, "gradient norm sum launch");
    }
    batches(gs, n, CLIP_SEGS, bs);
    for (auto& b : bs) {
        ClipArgs a;
        const double bytes = clip_args(b, a);
        a.no = no;
        const int grid = wgs_of(a.chunks, CLIP_WGS);
        rc = timed_launch(MU_K_CLIP, 0.0, bytes, s, [&] {
            if (nt) hipLaunchKernelGGL(k_clip<true>, dim3(grid), dim3(NTHR), 0, s, a);
            else hipLaunchKernelGGL(k_clip<false>, dim3(grid), dim3(NTHR), 0, s, a);
            return hipGetLastError();
        }, "clip launch");
        if (rc) return rc;
    }
    return MU_OK;
}

}  // namespace

extern "C" {

int mu_grad_norm_workspace_size(const mu_grad* gs, int32_t n, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check_list(gs, n, false, nullptr, nullptr);
        if (rc) return rc;
        std::vector<Batch> bs;
        batches(gs, n, SQ_SEGS, bs);
        *bytes = align_up(partials_of(bs) * sizeof(double));
        return MU_OK;
    });
}

int mu_grad_norm(const mu_grad* gs, int32_t n, float max_norm, float eps, float* norm_out, float* scale_out, void* ws,
                 size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        return norm_and_clip(gs, n, max_norm, eps, norm_out, scale_out, false, ws, ws_bytes, (hipStream_t)stream);
    });
}

int mu_clip_grads(const mu_grad* gs, int32_t n, float max_norm, float eps, float* norm_out, float* scale_out, void* ws,
                  size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        return norm_and_clip(gs, n, max_norm, eps, norm_out, scale_out, true, ws, ws_bytes, (hipStream_t)stream);
    });
}

}  // extern "C"
