// Embedding lookup and its gradient (gfx950): the C entry points and their
// kernels.
//
//   out[t, :]  = scale * weight[tokens[t], :]
//   grad[v, :] = scale * sum over t with tokens[t] == v, in rising t, of rows[t, :]
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

__device__ __forceinline__ int64_t token_at(const void* tokens, int bits, int64_t t) {
    return bits == 32 ? (int64_t)((const MU_GLOBAL int32_t*)tokens)[t] : ((const MU_GLOBAL int64_t*)tokens)[t];
}

template <typename T>
__global__ __launch_bounds__(NTHR) void k_lookup(mu_lookup E) {
    const int64_t t = blockIdx.x;
    const int64_t v = token_at(E.tokens, E.token_bits, t);
    const bool ok = v >= 0 && v < E.vocab;
    const MU_GLOBAL T* w = (const MU_GLOBAL T*)E.weight + (ok ? v : 0) * E.dim;
    MU_GLOBAL T* o = (MU_GLOBAL T*)E.out + t * E.dim;
    for (int64_t c = threadIdx.x; c < E.dim; c += NTHR) {
        if (ok && E.scale == 1.f) o[c] = w[c];
        else o[c] = from_f32<T>(ok ? E.scale * to_f32<T>(w[c]) : __builtin_nanf(""));
    }
}

template <typename TR, typename TG>
__global__ __launch_bounds__(NTHR) void k_rowgrad(mu_rowgrad E) {
    __shared__ int32_t tok[NTHR];
    const int64_t v = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * NTHR + threadIdx.x;
    float s = 0.f;
    for (int64_t t0 = 0; t0 < E.n_tokens && v != E.padding_idx; t0 += NTHR) {
        const int64_t t = t0 + threadIdx.x;
        int32_t id = -1;
        if (t < E.n_tokens) {
            const int64_t x = token_at(E.tokens, E.token_bits, t);
            if (x >= 0 && x < E.vocab) id = (int32_t)x;
        }
        tok[threadIdx.x] = id;
        if (!__syncthreads_or(id == (int32_t)v)) continue;
        if (c < E.dim)
            for (int j = 0; j < NTHR; ++j)
                if (tok[j] == (int32_t)v) s += to_f32<TR>(((const MU_GLOBAL TR*)E.rows)[(t0 + j) * E.dim + c]);
        __syncthreads();
    }
    if (c >= E.dim) return;
    MU_GLOBAL TG* g = (MU_GLOBAL TG*)E.grad + v * E.dim + c;
    float r = E.scale * s;
    if (E.accumulate) r += to_f32<TG>(*g);
    *g = from_f32<TG>(r);
}

size_t es_of(int dt) { return dt == MU_BF16 ? 2 : 4; }
bool known(int dt) { return dt == MU_F32 || dt == MU_BF16; }

int check_sizes(int64_t n_tokens, int64_t vocab, int64_t dim, int bits, float scale) {
    if (bits != 32 && bits != 64) return fail(MU_ERR_DTYPE, "token_bits must be 32 or 64 (got %d)", bits);
    if (n_tokens < 0 || n_tokens > 0x7fffffffLL) return fail(MU_ERR_INVALID_ARG, "n_tokens must be in [0, 2^31)");
    if (vocab < 1 || vocab > 0x7ffffffeLL) return fail(MU_ERR_INVALID_ARG, "vocab must be in [1, 2^31 - 1)");
    if (dim < 1 || dim > MU_MAX_DIM) return fail(MU_ERR_INVALID_ARG, "dim must be in [1, %d]", MU_MAX_DIM);
    if (!std::isfinite(scale)) return fail(MU_ERR_INVALID_ARG, "scale must be finite");
    return MU_OK;
}

Range range_of(const void* p, int64_t n, size_t es) { return {(uintptr_t)p, (uintptr_t)p + (size_t)n * es, 0}; }

int check_rowgrad(const mu_rowgrad* e) {
    if (!e) return fail(MU_ERR_INVALID_ARG, "argument is null");
    int rc = check_sizes(e->n_tokens, e->vocab, e->dim, e->token_bits, e->scale);
    if (rc) return rc;
    if (!known(e->row_dtype) || !known(e->grad_dtype)) return fail(MU_ERR_DTYPE, "unknown row or gradient dtype");
    if (e->accumulate != 0 && e->accumulate != 1) return fail(MU_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (e->padding_idx < -1 || e->padding_idx >= e->vocab)
        return fail(MU_ERR_INVALID_ARG, "padding_idx must be -1 or in [0, vocab)");
    return MU_OK;
}

}  // namespace

extern "C" {

int mu_embedding(const mu_lookup* e, void* stream) {
    return guarded([&]() -> int {
        if (!e) return fail(MU_ERR_INVALID_ARG, "argument is null");
        int rc = check_sizes(e->n_tokens, e->vocab, e->dim, e->token_bits, e->scale);
        if (rc) return rc;
        if (!known(e->dtype)) return fail(MU_ERR_DTYPE, "unknown dtype %d", e->dtype);
        if (e->n_tokens == 0) return MU_OK;
        if (!e->tokens || !e->weight || !e->out) return fail(MU_ERR_INVALID_ARG, "null tokens, weight or out");
        const size_t es = es_of(e->dtype);
        if (!aligned(e->tokens, e->token_bits / 8) || !aligned(e->weight, es) || !aligned(e->out, es))
            return fail(MU_ERR_LAYOUT, "misaligned buffer");
        std::vector<Range> in{range_of(e->out, e->n_tokens * e->dim, es), range_of(e->weight, e->vocab * e->dim, es)};
        std::vector<Range> tk{range_of(e->out, e->n_tokens * e->dim, es), range_of(e->tokens, e->n_tokens, e->token_bits / 8)};
        if (ranges_overlap(in) || ranges_overlap(tk)) return fail(MU_ERR_LAYOUT, "out overlaps an input");
        hipStream_t s = (hipStream_t)stream;
        const double bytes = (double)e->n_tokens * (2.0 * (double)e->dim * es + e->token_bits / 8);
        return timed_launch(MU_K_LOOKUP, 0.0, bytes, s, [&] {
            const dim3 grid((unsigned)e->n_tokens);
            if (e->dtype == MU_BF16) hipLaunchKernelGGL(k_lookup<bf16>, grid, dim3(NTHR), 0, s, *e);
            else hipLaunchKernelGGL(k_lookup<float>, grid, dim3(NTHR), 0, s, *e);
            return hipGetLastError();
        }, "embedding launch");
    });
}

int mu_embedding_grad_workspace_size(const mu_rowgrad* e, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check_rowgrad(e);
        if (rc) return rc;
        *bytes = 0;
        return MU_OK;
    });
}

int mu_embedding_grad(const mu_rowgrad* e, void* ws, size_t ws_bytes, void* stream) {
    (void)ws;
    (void)ws_bytes;
    return guarded([&]() -> int {
        int rc = check_rowgrad(e);
        if (rc) return rc;
        if (!e->grad || (e->n_tokens > 0 && (!e->tokens || !e->rows)))
            return fail(MU_ERR_INVALID_ARG, "null tokens, rows or grad");
        const size_t er = es_of(e->row_dtype), eg = es_of(e->grad_dtype);
        if (!aligned(e->tokens, e->token_bits / 8) || !aligned(e->rows, er) || !aligned(e->grad, eg))
            return fail(MU_ERR_LAYOUT, "misaligned buffer");
        std::vector<Range> a{range_of(e->grad, e->vocab * e->dim, eg), range_of(e->rows, e->n_tokens * e->dim, er)};
        std::vector<Range> b{range_of(e->grad, e->vocab * e->dim, eg), range_of(e->tokens, e->n_tokens, e->token_bits / 8)};
        if (e->n_tokens > 0 && (ranges_overlap(a) || ranges_overlap(b)))
            return fail(MU_ERR_LAYOUT, "grad overlaps an input");
        if (e->n_tokens == 0 && e->accumulate) return MU_OK;
        hipStream_t s = (hipStream_t)stream;
        const double bytes = (double)e->n_tokens * ((double)e->dim * er + e->token_bits / 8) + (double)e->vocab * e->dim * eg;
        return timed_launch(MU_K_ROWGRAD, 0.0, bytes, s, [&] {
            const dim3 grid((unsigned)e->vocab, (unsigned)((e->dim + NTHR - 1) / NTHR)), block(NTHR);
            if (e->row_dtype == MU_BF16) {
                if (e->grad_dtype == MU_BF16) hipLaunchKernelGGL((k_rowgrad<bf16, bf16>), grid, block, 0, s, *e);
                else hipLaunchKernelGGL((k_rowgrad<bf16, float>), grid, block, 0, s, *e);
            } else {
                if (e->grad_dtype == MU_BF16) hipLaunchKernelGGL((k_rowgrad<float, bf16>), grid, block, 0, s, *e);
                else hipLaunchKernelGGL((k_rowgrad<float, float>), grid, block, 0, s, *e);
            }
            return hipGetLastError();
        }, "embedding gradient launch");
    });
}

}  // extern "C"
