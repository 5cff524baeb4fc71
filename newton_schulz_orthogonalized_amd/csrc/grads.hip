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

// Vectors at element alignment: gfx950 takes global vector accesses at any
// address, so tensors that start anywhere in an allocation need no other path.
typedef bf16x8 bf16x8u __attribute__((aligned(2)));
typedef f32x4 f32x4u __attribute__((aligned(4)));

template <typename T>
__device__ __forceinline__ void load8(const MU_GLOBAL T* p, float v[8]) {
    if constexpr (sizeof(T) == 2) {
        const bf16x8 q = *(const MU_GLOBAL bf16x8u*)p;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)q[e];
    } else {
        const f32x4 a = *(const MU_GLOBAL f32x4u*)p, b = *(const MU_GLOBAL f32x4u*)(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[e + 4] = b[e]; }
    }
}
template <typename T>
__device__ __forceinline__ void store8(MU_GLOBAL T* p, const float v[8]) {
    if constexpr (sizeof(T) == 2) {
        bf16x8 q;
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = (bf16)v[e];
        *(MU_GLOBAL bf16x8u*)p = q;
    } else {
        *(MU_GLOBAL f32x4u*)p = f32x4{v[0], v[1], v[2], v[3]};
        *(MU_GLOBAL f32x4u*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
}

__device__ __forceinline__ double block_sum(double v, double* red) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const double s = ((red[0] + red[1]) + red[2]) + red[3];
    __syncthreads();
    return s;
}

template <typename T>
__device__ double sumsq_chunk(const void* base, int64_t i0, int64_t n) {
    const MU_GLOBAL T* p = (const MU_GLOBAL T*)base;
    double s = 0.0;
    for (int64_t i = i0 + threadIdx.x * 8; i < min<int64_t>(n, i0 + GRAD_CHUNK); i += NTHR * 8) {
        float v[8];
        if (i + 8 <= n) load8<T>(p + i, v);
        else
            for (int e = 0; e < 8; ++e) v[e] = i + e < n ? to_f32<T>(p[i + e]) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
    }
    return s;
}

__global__ __launch_bounds__(NTHR) void k_sumsq(SqArgs A) {
    __shared__ double red[4];
    double s = 0.0;
    int i = 0;
    for (int c = blockIdx.x; c < A.chunks; c += gridDim.x) {
        while (i + 1 < A.nseg && A.seg[i + 1].c0 <= c) ++i;
        const int64_t i0 = (int64_t)(c - A.seg[i].c0) * GRAD_CHUNK;
        if (A.seg[i].dtype == DT_BF16) s += sumsq_chunk<bf16>(A.seg[i].p, i0, A.seg[i].n);
        else s += sumsq_chunk<float>(A.seg[i].p, i0, A.seg[i].n);
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0) gp(A.partials)[blockIdx.x] = s;
}

// The sum of the partials in a fixed order, by every thread of a workgroup;
// norm and c are written by the workgroup that `writes`. Returns c.
__device__ float finish_norm(const NormOut& N, bool writes, double* red) {
    double s = 0.0;
    for (int i = threadIdx.x; i < N.n; i += NTHR) s += gp(N.partials)[i];
    s = block_sum(s, red);
    const double norm = sqrt(s);
    const double r = (double)N.max_norm / (norm + (double)N.eps);
    // 0 / 0 (both bounds 0 and no gradient) clips nothing; a NaN norm stays NaN
    const float c = isnan(norm) ? (float)norm : (r < 1.0 ? (float)r : 1.f);
    if (writes && threadIdx.x == 0) {
        if (N.norm) *gp(N.norm) = (float)norm;
        if (N.scale) *gp(N.scale) = c;
    }
    return c;
}

__global__ __launch_bounds__(NTHR) void k_norm_final(NormOut N) {
    __shared__ double red[4];
    finish_norm(N, true, red);
}

template <typename TI, typename TO>
__device__ void clip_chunk(const void* base, void* out, int64_t i0, int64_t n, float c) {
    const MU_GLOBAL TI* p = (const MU_GLOBAL TI*)base;
    MU_GLOBAL TO* o = (MU_GLOBAL TO*)out;
    for (int64_t i = i0 + threadIdx.x * 8; i < min<int64_t>(n, i0 + GRAD_CHUNK); i += NTHR * 8) {
        if (i + 8 <= n) {
            float v[8];
            load8<TI>(p + i, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= c;
            store8<TO>(o + i, v);
        } else {
            for (int64_t j = i; j < n; ++j) o[j] = from_f32<TO>(c * to_f32<TI>(p[j]));
        }
    }
}

__global__ __launch_bounds__(NTHR) void k_clip(ClipArgs A) {
    __shared__ double red[4];
    const float c = finish_norm(A.no, blockIdx.x == 0, red);
    int i = 0;
    for (int q = blockIdx.x; q < A.chunks; q += gridDim.x) {
        while (i + 1 < A.nseg && A.seg[i + 1].c0 <= q) ++i;
        const ClipSeg& S = A.seg[i];
        if (c == 1.f && S.p == S.out) continue;   // in place and nothing to clip
        const int64_t i0 = (int64_t)(q - S.c0) * GRAD_CHUNK;
        if (S.dtype == DT_BF16) {
            if (S.out_dtype == DT_BF16) clip_chunk<bf16, bf16>(S.p, S.out, i0, S.n, c);
            else clip_chunk<bf16, float>(S.p, S.out, i0, S.n, c);
        } else {
            if (S.out_dtype == DT_BF16) clip_chunk<float, bf16>(S.p, S.out, i0, S.n, c);
            else clip_chunk<float, float>(S.p, S.out, i0, S.n, c);
        }
    }
}

size_t es_of(int dt) { return dt == MU_BF16 ? 2 : 4; }

int check_list(const mu_grad* gs, int32_t n, bool with_out) {
    if (n < 0) return fail(MU_ERR_INVALID_ARG, "n must be >= 0");
    if (n > 0 && !gs) return fail(MU_ERR_INVALID_ARG, "gradient list is null");
    std::vector<Range> ranges;
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

// Launches of at most `segs` tensors and 2^31 - 1 chunks each: fn(first list
// entry's index in `order`, count, chunks).
struct Batch {
    std::vector<int> items;
    int64_t chunks = 0;
};
int batches(const mu_grad* gs, int32_t n, int segs, std::vector<Batch>& out) {
    out.clear();
    for (int i = 0; i < n; ++i) {
        if (gs[i].numel == 0) continue;
        const int64_t c = chunks_of(gs[i].numel);
        if (c > 0x3fffffff) return fail(MU_ERR_INVALID_ARG, "gradient %d is too large for one launch", i);
        if (out.empty() || (int)out.back().items.size() == segs || out.back().chunks + c > 0x3fffffff) out.emplace_back();
        out.back().items.push_back(i);
        out.back().chunks += c;
    }
    return MU_OK;
}

size_t partials_of(const std::vector<Batch>& b) {
    size_t p = 0;
    for (auto& x : b) p += (size_t)std::min<int64_t>(x.chunks, SQ_WGS);
    return p;
}

int norm_and_clip(const mu_grad* gs, int32_t n, float max_norm, float eps, float* norm_out, float* scale_out, bool clip,
                  void* ws, size_t ws_bytes, hipStream_t s) {
    int rc = check_list(gs, n, clip);
    if (rc) return rc;
    if (!(max_norm >= 0.f)) return fail(MU_ERR_INVALID_ARG, "max_norm must be >= 0");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(MU_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!clip && !norm_out && !scale_out) return fail(MU_ERR_INVALID_ARG, "norm_out and scale_out are both null");
    if (!aligned(norm_out, 4) || !aligned(scale_out, 4)) return fail(MU_ERR_LAYOUT, "misaligned norm_out or scale_out");
    std::vector<Batch> bs;
    rc = batches(gs, n, SQ_SEGS, bs);
    if (rc) return rc;
    const size_t np = partials_of(bs), need = align_up(np * sizeof(double));
    if (np) {
        if (!ws) return fail(MU_ERR_WORKSPACE, "workspace is null (need %zu bytes)", need);
        if (!aligned(ws, ALIGN)) return fail(MU_ERR_WORKSPACE, "workspace must be 256-byte aligned");
        if (ws_bytes < need) return fail(MU_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    }
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
        const int grid = (int)std::min<int64_t>(c, SQ_WGS);
        part += grid;
        rc = timed_launch(MU_K_GRADNORM, 0.0, bytes, s, [&] {
            hipLaunchKernelGGL(k_sumsq, dim3(grid), dim3(NTHR), 0, s, a);
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
    rc = batches(gs, n, CLIP_SEGS, bs);
    if (rc) return rc;
    for (auto& b : bs) {
        ClipArgs a;
        double bytes = 0;
        int64_t c = 0;
        a.no = no;
        a.nseg = (int)b.items.size();
        for (int k = 0; k < a.nseg; ++k) {
            const mu_grad& g = gs[b.items[k]];
            a.seg[k] = ClipSeg{g.grad, g.out, g.numel, (int32_t)c, (int16_t)g.dtype, (int16_t)g.out_dtype};
            c += chunks_of(g.numel);
            bytes += (double)g.numel * (es_of(g.dtype) + es_of(g.out_dtype));
        }
        a.chunks = (int)c;
        const int grid = (int)std::min<int64_t>(c, SQ_WGS);
        rc = timed_launch(MU_K_CLIP, 0.0, bytes, s, [&] {
            hipLaunchKernelGGL(k_clip, dim3(grid), dim3(NTHR), 0, s, a);
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
        int rc = check_list(gs, n, false);
        if (rc) return rc;
        std::vector<Batch> bs;
        rc = batches(gs, n, SQ_SEGS, bs);
        if (rc) return rc;
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
