// The largest attention logit magnitude of each query head (gfx950): the C
// entry point and its kernels.
//
//   max_logit[h] = |scale| * max over b and visible (i, j) of |q[b,i,h,:] . k[b,j,h/G,:]|
//
// The maximum does not depend on the order in which pairs are taken, so
// workgroups join their maxima with an atomic and the result is the same
// bits every time. It is taken over the float bits of the magnitudes: for
// values without a sign they order as integers, with NaN above infinity.
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

__global__ __launch_bounds__(NTHR) void k_qk_init(float* out, int n) {
    for (int i = threadIdx.x; i < n; i += NTHR) gp(out)[i] = 0.f;
}

struct Seq {
    int64_t q0, k0;   // element offset of its first row (without the head)
    int64_t nq, nk;
};

__device__ inline int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

__device__ inline Seq seq_of(const mu_qk_logits& A, int b) {
    Seq s;
    if (A.cu_q) {
        const MU_GLOBAL int32_t* cq = (const MU_GLOBAL int32_t*)A.cu_q;
        const MU_GLOBAL int32_t* ck = A.cu_k ? (const MU_GLOBAL int32_t*)A.cu_k : cq;
        const int64_t a = clamp64(cq[b], 0, A.q_len), c = clamp64(ck[b], 0, A.k_len);
        s.nq = clamp64(cq[b + 1], a, A.q_len) - a;
        s.nk = clamp64(ck[b + 1], c, A.k_len) - c;
        s.q0 = a * A.q_stride_s;
        s.k0 = c * A.k_stride_s;
    } else {
        s.nq = A.q_lengths ? clamp64(((const MU_GLOBAL int32_t*)A.q_lengths)[b], 0, A.q_len) : A.q_len;
        s.nk = A.k_lengths ? clamp64(((const MU_GLOBAL int32_t*)A.k_lengths)[b], 0, A.k_len) : A.k_len;
        s.q0 = b * A.q_stride_b;
        s.k0 = b * A.k_stride_b;
    }
    return s;
}

// One query of one sequence and head a workgroup, one key a thread at a time.
template <typename T>
__global__ __launch_bounds__(NTHR) void k_qkmax(mu_qk_logits A) {
    __shared__ float qs[MU_QK_MAX_DIM];
    __shared__ int red[4];
    const int h = blockIdx.y, b = blockIdx.z;
    const Seq S = seq_of(A, b);
    const int64_t i = blockIdx.x;
    if (i >= S.nq) return;
    const MU_GLOBAL T* q = (const MU_GLOBAL T*)A.q + S.q0 + i * A.q_stride_s + h * A.q_stride_h;
    const MU_GLOBAL T* k = (const MU_GLOBAL T*)A.k + S.k0 + (h / (A.q_heads / A.k_heads)) * A.k_stride_h;
    for (int d = threadIdx.x; d < A.dim; d += NTHR) qs[d] = to_f32<T>(q[d]);
    __syncthreads();
    const int64_t last = A.causal ? min<int64_t>(S.nk, i + S.nk - S.nq + 1) : S.nk;
    int best = 0;
    for (int64_t j = threadIdx.x; j < last; j += NTHR) {
        float s = 0.f;
        for (int d = 0; d < A.dim; ++d) s = fmaf(qs[d], to_f32<T>(k[j * A.k_stride_s + d]), s);
        best = max(best, __float_as_int(s) & 0x7fffffff);
    }
    for (int off = 32; off >= 1; off >>= 1) best = max(best, __shfl_xor(best, off, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
        best = max(max(red[0], red[1]), max(red[2], red[3]));
        atomicMax((int*)A.max_logit + h, __float_as_int(fabsf(A.scale) * __int_as_float(best)) & 0x7fffffff);
    }
}

int check(const mu_qk_logits* a) {
    if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
    if (a->dtype != MU_F32 && a->dtype != MU_BF16) return fail(MU_ERR_DTYPE, "unknown dtype %d", a->dtype);
    if (a->batch < 0 || a->batch > 65535 || a->q_len < 0 || a->k_len < 0 || a->q_len > 0x7fffff00LL || a->k_len > 0x7fffff00LL)
        return fail(MU_ERR_INVALID_ARG, "bad batch or length");
    if (a->q_heads < 1 || a->q_heads > 65535 || a->k_heads < 1 || a->q_heads % a->k_heads != 0)
        return fail(MU_ERR_INVALID_ARG, "head counts must be >= 1 and k_heads divide q_heads");
    if (a->dim < 1 || a->dim > MU_QK_MAX_DIM) return fail(MU_ERR_INVALID_ARG, "dim must be in [1, %d]", MU_QK_MAX_DIM);
    if ((a->causal != 0 && a->causal != 1) || (a->accumulate != 0 && a->accumulate != 1))
        return fail(MU_ERR_INVALID_ARG, "causal and accumulate must be 0 or 1");
    if (!std::isfinite(a->scale)) return fail(MU_ERR_INVALID_ARG, "scale must be finite");
    if (a->q_stride_b < 0 || a->q_stride_s < 0 || a->q_stride_h < 0 || a->k_stride_b < 0 || a->k_stride_s < 0 || a->k_stride_h < 0)
        return fail(MU_ERR_INVALID_ARG, "strides must be >= 0");
    if (!a->max_logit) return fail(MU_ERR_INVALID_ARG, "max_logit is null");
    if (a->cu_q && (a->q_lengths || a->k_lengths)) return fail(MU_ERR_INVALID_ARG, "packed sequences take no lengths");
    if (!a->cu_q && a->cu_k) return fail(MU_ERR_INVALID_ARG, "cu_k without cu_q");
    if (a->cu_q && !a->cu_k && a->q_len != a->k_len)
        return fail(MU_ERR_INVALID_ARG, "one cu for both needs as many query as key rows");
    const size_t es = a->dtype == MU_BF16 ? 2 : 4;
    if (!aligned(a->q, es) || !aligned(a->k, es) || !aligned(a->max_logit, 4) || !aligned(a->q_lengths, 4) ||
        !aligned(a->k_lengths, 4) || !aligned(a->cu_q, 4) || !aligned(a->cu_k, 4))
        return fail(MU_ERR_LAYOUT, "misaligned buffer");
    if (a->batch > 0 && a->q_len > 0 && a->k_len > 0 && (!a->q || !a->k)) return fail(MU_ERR_INVALID_ARG, "q or k is null");
    return MU_OK;
}

}  // namespace

extern "C" {

int mu_qk_max_logits(const mu_qk_logits* a, void* stream) {
    return guarded([&]() -> int {
        int rc = check(a);
        if (rc) return rc;
        hipStream_t s = (hipStream_t)stream;
        if (!a->accumulate) {
            rc = timed_launch(MU_K_QKMAX, 0.0, 4.0 * a->q_heads, s, [&] {
                hipLaunchKernelGGL(k_qk_init, dim3(1), dim3(NTHR), 0, s, a->max_logit, a->q_heads);
                return hipGetLastError();
            }, "max logits init");
            if (rc) return rc;
        }
        if (a->batch == 0 || a->q_len == 0 || a->k_len == 0) return MU_OK;
        const double es = a->dtype == MU_BF16 ? 2 : 4, nb = a->cu_q ? 1 : a->batch;
        const double bytes = nb * a->dim * es * ((double)a->q_len * a->q_heads + (double)a->k_len * a->k_heads);
        const double flops = 2.0 * nb * (double)a->q_len * (double)a->k_len * a->q_heads * a->dim * (a->causal ? 0.5 : 1.0);
        return timed_launch(MU_K_QKMAX, flops, bytes, s, [&] {
            const dim3 grid((unsigned)a->q_len, (unsigned)a->q_heads, (unsigned)a->batch);
            if (a->dtype == MU_BF16) hipLaunchKernelGGL(k_qkmax<bf16>, grid, dim3(NTHR), 0, s, *a);
            else hipLaunchKernelGGL(k_qkmax<float>, grid, dim3(NTHR), 0, s, *a);
            return hipGetLastError();
        }, "max logits launch");
    });
}

}  // extern "C"
