// The gated feed-forward block (gfx950): the C entry points and their kernels.
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) * u
//   dg = dh * u * act'(g),  du = dh * act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// One tiled product with four uses:
//   FWD     x times both weights; a tile holds the same columns of g and u, so the
//           activation, the product (and g and u, where the gradient wants them)
//           leave from registers and no other pass exists
//   RECOMP  the same products again in the backward pass, whose epilogue reads dh
//           and leaves dg and du
//   DX      one product over 2 * hidden: dg with Wg, then du with Wu
//   DW      both weight gradients over the tokens, one launch
// Operands are read in their own layouts: with k along the rows (x and the weights
// in FWD, dg and du in DX) or k down the rows (the weights in DX; dg, du and x in
// DW), whose bfloat16 fragments come out of LDS through ds_read_b64_tr_b16. No
// transposed copy exists. Rows that do not start at 16-byte steps (odd dim) are
// copied into the workspace with padded rows first.
//
// Slices of 128 bytes of k (64 bfloat16, 32 float32) move from memory to LDS with
// direct loads, 1 KB each; what lies outside an operand reads as zero.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/muon_mi355x.h"
#include "capi_common.hpp"
#include "common.hpp"
#include "gated.hpp"
#include "vec.hpp"

using namespace mu;

using namespace mu::gated;

namespace {

constexpr int TILE = 128;   // tile edge
#define MU_WAIT_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (15 << 8) | (((n) >> 4) << 14))

template <typename T, int MODE, int TS>
__global__ __launch_bounds__(NTHR, TS == 256 ? 1 : 2) void k_tile(TileArgs A) {
    constexpr bool DUAL = MODE == FWD || MODE == RECOMP;
    constexpr int ES = sizeof(T), BK = bk<T>(), WT = TS / 2, F = WT / 16, TN = DUAL ? TS / 2 : TS;
    typedef Operand<T, TS, MODE == DW> OA;
    typedef Operand<T, TS, MODE == DX || MODE == DW> OB;
    __shared__ __attribute__((aligned(1024))) char sA0[TS * 128];
    __shared__ __attribute__((aligned(1024))) char sA1[TS * 128];
    __shared__ __attribute__((aligned(1024))) char sB0[TS * 128];
    __shared__ __attribute__((aligned(1024))) char sB1[TS * 128];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int total = A.tiles_m * A.tiles_n;
    int t = xcd_remap(blockIdx.x, gridDim.x);
    if (t >= total) return;
    int ti, tj;
    tile_of(t, A.tiles_m, A.tiles_n, ti, tj);
    int which = 0;   // DW: the gate's gradient, then the up projection's
    if (MODE == DW && ti >= A.tiles_m / 2) {
        which = 1;
        ti -= A.tiles_m / 2;
    }
    const int64_t m0 = (int64_t)ti * TS, n0 = (int64_t)tj * TN;
    const int kth = (int)((A.k + BK - 1) / BK), kts = MODE == DX ? 2 * kth : kth;
    const int kt0 = blockIdx.y * A.kt_split, kt1 = min(kts, kt0 + A.kt_split);

    // Direct loads of slice kt into a slot.
    auto dma = [&](char* sa, char* sb, int kt) {
        const int seg = MODE == DX && kt >= kth ? 1 : 0;
        const int64_t k0 = (int64_t)(kt - seg * kth) * BK;
        {
            const char* base = (const char*)A.a[MODE == DX ? seg : which];
            __amdgpu_buffer_rsrc_t ra;
            if (MODE == DW) ra = resource(base + (k0 * A.lda + m0) * ES, ((A.k - k0) * A.lda - m0) * ES);
            else ra = resource(base + (m0 * A.lda + k0) * ES, ((A.m - m0) * A.lda - k0) * ES);
#pragma unroll
            for (int i = 0; i < OA::NI; ++i) {
                const int row = OA::lds_row(i, wave, lane), c = OA::chunk(row, lane);
                int off = row * (int)A.lda * ES + c * 16;
                if (MODE != DW && k0 + c * (16 / ES) >= A.k) off = OUTSIDE;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDSP void*)(sa + (i * 4 + wave) * 1024), 16, off, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < OB::NI; ++i) {
            const int row = OB::lds_row(i, wave, lane), c = OB::chunk(row, lane);
            __amdgpu_buffer_rsrc_t rb;
            int off;
            if constexpr (DUAL) {
                // LDS rows: for each half of the columns, those of the gate and of the up projection
                const int r0 = i * 32 + wave * 8, half = r0 / WT, in = r0 % WT, part = in / (WT / 2);
                const int64_t f0 = n0 + half * (WT / 2) + in % (WT / 2);
                rb = resource((const char*)A.b[part] + (f0 * A.ldb + k0) * ES, ((A.n - f0) * A.ldb - k0) * ES);
                off = (lane >> 3) * (int)A.ldb * ES + c * 16;
                if (k0 + c * (16 / ES) >= A.k) off = OUTSIDE;
            } else {
                rb = resource((const char*)A.b[MODE == DX ? seg : 0] + (k0 * A.ldb + n0) * ES, ((A.k - k0) * A.ldb - n0) * ES);
                off = row * (int)A.ldb * ES + c * 16;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LDSP void*)(sb + (i * 4 + wave) * 1024), 16, off, 0, 0, 0);
        }
    };

    const int wm = (wave >> 1) * WT, wn = (wave & 1) * WT;
    f32x4 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (the weights' side first: a lane then holds four consecutive columns of a row)
    auto compute = [&](const char* sa, const char* sb) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            typename Mma<T>::Frag af[F], bf[F];
#pragma unroll
            for (int f = 0; f < F; ++f) bf[f] = OB::read(sb, wn, f, kk, lane);
#pragma unroll
            for (int f = 0; f < F; ++f) af[f] = OA::read(sa, wm, f, kk, lane);
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int j = 0; j < F; ++j) acc[i][j] = mma(bf[j], af[i], acc[i][j]);
        }
    };
    if (kt0 < kt1) dma(sA0, sB0, kt0);
    for (int kt = kt0; kt < kt1; kt += 2) {
        MU_WAIT_VMCNT(0);
        __syncthreads();
        if (kt + 1 < kt1) dma(sA1, sB1, kt + 1);
        compute(sA0, sB0);
        if (kt + 1 >= kt1) break;
        MU_WAIT_VMCNT(0);
        __syncthreads();
        if (kt + 2 < kt1) dma(sA0, sB0, kt + 2);
        compute(sA1, sB1);
    }

    // Lane l holds columns 16 j + 4 (l >> 4) .. +3 of row 16 i + (l & 15) of each fragment.
    constexpr bool FAST = ES == 2;
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int64_t row = m0 + wm + i * 16 + (lane & 15);
        if (row >= A.m) continue;
        if constexpr (DUAL) {
#pragma unroll
            for (int j = 0; j < F / 2; ++j) {
                const int64_t col = n0 + wn / 2 + j * 16 + 4 * (lane >> 4);
                // (RECOMP also writes the zeros behind its padded rows, which DX reads)
                const int cnt = (int)min((int64_t)4, A.n - col);
                const int put = MODE == RECOMP ? (int)min((int64_t)4, A.ldo - col) : cnt;
                if (put <= 0) continue;
                const f32x4 g = acc[i][j], u = acc[i][j + F / 2];
                float o0[4], o1[4];
                if constexpr (MODE == FWD) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a, s;
                        act_of<FAST>(A.act, g[e], a, s);
                        o0[e] = a * u[e];
                    }
                    for (int e = 0; e < cnt; ++e) ((MU_GLOBAL T*)A.out[0])[row * A.ldo + col + e] = from_f32<T>(o0[e]);
                    if (A.gates[0])
                        for (int e = 0; e < cnt; ++e) {
                            ((MU_GLOBAL T*)A.gates[0])[row * A.ldo + col + e] = from_f32<T>(g[e]);
                            ((MU_GLOBAL T*)A.gates[1])[row * A.ldo + col + e] = from_f32<T>(u[e]);
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float d = e < cnt ? to_f32<T>(((const MU_GLOBAL T*)A.dh)[row * A.n + col + e]) : 0.f;
                        float a, s;
                        act_of<FAST>(A.act, g[e], a, s);
                        o0[e] = d * u[e] * s;
                        o1[e] = d * a;
                    }
                    for (int e = 0; e < put; ++e) {
                        ((MU_GLOBAL T*)A.out[0])[row * A.ldo + col + e] = from_f32<T>(o0[e]);
                        ((MU_GLOBAL T*)A.out[1])[row * A.ldo + col + e] = from_f32<T>(o1[e]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < F; ++j) {
                const int64_t col = n0 + wn + j * 16 + 4 * (lane >> 4);
                const int cnt = (int)min((int64_t)4, A.n - col);
                if (cnt <= 0) continue;
                const int64_t at = row * A.n + col;
                if (A.part) {
                    float* p = A.part + ((int64_t)blockIdx.y * (MODE == DW ? 2 : 1) + which) * A.m * A.n + at;
                    for (int e = 0; e < cnt; ++e) gp(p)[e] = acc[i][j][e];
                } else if (MODE == DW && (A.out_f32 || ES == 4)) {
                    MU_GLOBAL float* p = (MU_GLOBAL float*)A.out[which] + at;
                    for (int e = 0; e < cnt; ++e) p[e] = acc[i][j][e] + (A.accumulate ? p[e] : 0.f);
                } else {
                    MU_GLOBAL T* p = (MU_GLOBAL T*)A.out[which] + at;
                    for (int e = 0; e < cnt; ++e) p[e] = from_f32<T>(acc[i][j][e] + (A.accumulate ? to_f32<T>(p[e]) : 0.f));
                }
            }
        }
    }
}

// Sums of the splits' results, in order.
struct JoinArgs {
    const float* part;
    void* out[2];
    int64_t n;        // elements of a result
    int splits, nout;
    bool out_f32, accumulate;
};
__global__ __launch_bounds__(NTHR) void k_join(JoinArgs A) {
    const int64_t i = (int64_t)blockIdx.x * NTHR + threadIdx.x;
    if (i >= A.n * A.nout) return;
    const int which = i >= A.n;
    const int64_t at = i - which * A.n;
    float s = 0.f;
    for (int k = 0; k < A.splits; ++k) s += gp(A.part)[(int64_t)k * A.nout * A.n + i];
    if (A.out_f32) {
        MU_GLOBAL float* o = (MU_GLOBAL float*)A.out[which] + at;
        *o = A.accumulate ? *o + s : s;
    } else {
        MU_GLOBAL bf16* o = (MU_GLOBAL bf16*)A.out[which] + at;
        *o = (bf16)(A.accumulate ? (float)*o + s : s);
    }
}

// dg and du from the saved g and u: rows of `n`, into rows of `pitch`, zeros behind.
struct SlopeArgs {
    const void *dh, *g, *u;
    void *dg, *du;
    int64_t rows, n, pitch;
    int act;
};
template <typename T>
__global__ __launch_bounds__(NTHR) void k_slopes(SlopeArgs A) {
    constexpr int V = vec_of<T>();
    const int64_t runs = A.pitch / V, total = A.rows * runs;
    for (int64_t i = (int64_t)blockIdx.x * NTHR + threadIdx.x; i < total; i += (int64_t)gridDim.x * NTHR) {
        const int64_t row = i / runs, c = (i - row * runs) * V, at = row * A.n + c;
        const int cnt = (int)min((int64_t)V, A.n - c);
        float d[V], g[V], u[V];
        load_run<T, V>((const T*)A.dh + at, cnt, d);
        load_run<T, V>((const T*)A.g + at, cnt, g);
        load_run<T, V>((const T*)A.u + at, cnt, u);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float a, s;
            act_of<sizeof(T) == 2>(A.act, g[e], a, s);
            g[e] = e < cnt ? d[e] * u[e] * s : 0.f;
            u[e] = e < cnt ? d[e] * a : 0.f;
        }
        store_run<T, V>((T*)A.dg + row * A.pitch + c, V, g);
        store_run<T, V>((T*)A.du + row * A.pitch + c, V, u);
    }
}

// Rows of n elements into rows of `pitch`, zeros behind them.
struct PackArgs {
    const void* src;
    void* dst;
    int64_t rows, n, pitch;
};
template <typename T>
__global__ __launch_bounds__(NTHR) void k_pack(PackArgs A) {
    constexpr int V = vec_of<T>();
    const int64_t runs = A.pitch / V, total = A.rows * runs;
    for (int64_t i = (int64_t)blockIdx.x * NTHR + threadIdx.x; i < total; i += (int64_t)gridDim.x * NTHR) {
        const int64_t row = i / runs, c = (i - row * runs) * V;
        float v[V];
        load_run<T, V>((const T*)A.src + row * A.n + c, (int)min((int64_t)V, A.n - c), v);
        store_run<T, V>((T*)A.dst + row * A.pitch + c, V, v);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
size_t es_of(int dtype) { return dtype == MU_BF16 ? 2 : 4; }
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An operand: where it lies, or the place of its padded copy in the workspace.
struct Source {
    const void* p;
    int64_t rows, n, pitch;
    bool copied;
    size_t off;
};

struct Plan {
    Source x, wg, wu;
    size_t off_dg, off_du, off_part, bytes;
    int64_t pitch_h;                    // of dg and du
    int kt_dx, splits_dx, kt_dw, splits_dw;
};

Source source(const void* p, int64_t rows, int64_t n, int es, Plan& pl) {
    const int64_t v = 16 / es;
    Source s{p, rows, n, n, n % v != 0 || !aligned(p, 16), 0};
    if (s.copied) {
        s.pitch = round_up(n, v);
        s.off = pl.bytes;
        pl.bytes += align_up((size_t)(rows * s.pitch) * es);
    }
    return s;
}

// Splits of k where the tiles alone leave most of the chip idle.
void split_k(int64_t tiles, int64_t kts, int& kt, int& splits) {
    splits = 1;
    if (tiles < 256) splits = (int)std::max<int64_t>(1, std::min<int64_t>({512 / tiles, kts / 8, 16}));
    kt = (int)ceil_div(kts, splits);
    splits = (int)std::max<int64_t>(1, ceil_div(kts, kt));
}

Plan plan_fwd(const mu_gated* a) {
    Plan p{};
    const int es = (int)es_of(a->dtype);
    p.x = source(a->x, a->tokens, a->dim, es, p);
    p.wg = source(a->w_gate, a->hidden, a->dim, es, p);
    p.wu = source(a->w_up, a->hidden, a->dim, es, p);
    return p;
}

Plan plan_bwd(const mu_gated_grad* a) {
    Plan p{};
    const int es = (int)es_of(a->dtype);
    const bool again = !a->gate;
    p.x = {a->x, a->tokens, a->dim, a->dim, false, 0};
    p.wg = {a->w_gate, a->hidden, a->dim, a->dim, false, 0};
    p.wu = {a->w_up, a->hidden, a->dim, a->dim, false, 0};
    if (again || a->d_gate) p.x = source(a->x, a->tokens, a->dim, es, p);
    if (again || a->dx) {
        p.wg = source(a->w_gate, a->hidden, a->dim, es, p);
        p.wu = source(a->w_up, a->hidden, a->dim, es, p);
    }
    p.pitch_h = round_up(a->hidden, 16 / es);
    p.off_dg = p.bytes;
    p.bytes += align_up((size_t)(a->tokens * p.pitch_h) * es);
    p.off_du = p.bytes;
    p.bytes += align_up((size_t)(a->tokens * p.pitch_h) * es);
    const int64_t bk = 128 / es;
    split_k(ceil_div(a->tokens, TILE) * ceil_div(a->dim, TILE), 2 * ceil_div(a->hidden, bk), p.kt_dx, p.splits_dx);
    split_k(2 * ceil_div(a->hidden, TILE) * ceil_div(a->dim, TILE), ceil_div(a->tokens, bk), p.kt_dw, p.splits_dw);
    size_t part = 0;
    if (a->dx && p.splits_dx > 1) part = sizeof(float) * (size_t)(p.splits_dx * a->tokens * a->dim);
    if (a->d_gate && p.splits_dw > 1) part = std::max(part, sizeof(float) * (size_t)(p.splits_dw * 2 * a->hidden * a->dim));
    p.off_part = p.bytes;
    p.bytes += align_up(part);
    return p;
}

const void* at(const Source& s, const char* ws) { return s.copied ? ws + s.off : s.p; }

template <typename T>
int pack(int kernel, const Source& s, char* ws, hipStream_t st) {
    if (!s.copied || s.rows == 0) return MU_OK;
    return timed_launch(kernel, 0.0, 0.0, st, [&] {
        const int64_t wgs = ceil_div(s.rows * (s.pitch / vec_of<T>()), NTHR);
        hipLaunchKernelGGL(k_pack<T>, dim3((unsigned)std::min<int64_t>(wgs, 1 << 16)), dim3(NTHR), 0, st,
                           PackArgs{s.p, ws + s.off, s.rows, s.n, s.pitch});
        return hipGetLastError();
    }, "operand copy launch");
}

template <typename T, int MODE>
int product(int kernel, TileArgs a, int splits, double flops, double bytes, hipStream_t s) {
    if (sizeof(T) == 2 && splits == 1) {
        const int64_t tm = ceil_div(a.m, 256) * (MODE == DW ? 2 : 1), tn = ceil_div(a.n, MODE == FWD || MODE == RECOMP ? 128 : 256);
        if (tm * tn >= 224 && tm * tn <= (1 << 23)) {
            a.tiles_m = (int)tm;
            a.tiles_n = (int)tn;
            a.aligned = a.n % 8 == 0 && a.ldo % 8 == 0;
            for (const void* p : {(const void*)a.out[0], (const void*)a.out[1], (const void*)a.gates[0], (const void*)a.gates[1]})
                a.aligned = a.aligned && aligned(p, 16);
            return timed_launch(kernel, flops, bytes, s, [&] {
                return launch_wide(MODE, a, (int)std::min<int64_t>(256, round_up(tm * tn, 8)), s);
            }, "gated feed-forward product launch");
        }
    }
    const int64_t tm = ceil_div(a.m, TILE) * (MODE == DW ? 2 : 1), tn = ceil_div(a.n, MODE == FWD || MODE == RECOMP ? TILE / 2 : TILE);
    if (tm * tn > (1 << 23)) return fail(MU_ERR_INVALID_ARG, "too many tiles for one launch");
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    return timed_launch(kernel, flops, bytes, s, [&] {
        const dim3 grid((unsigned)round_up(tm * tn, 8), (unsigned)splits);
        hipLaunchKernelGGL((k_tile<T, MODE, TILE>), grid, dim3(NTHR), 0, s, a);
        return hipGetLastError();
    }, "gated feed-forward product launch");
}

int join(JoinArgs j, hipStream_t s) {
    const int64_t wgs = ceil_div(j.n * j.nout, NTHR);
    if (wgs > (1 << 24) - 1) return fail(MU_ERR_INVALID_ARG, "too many elements for one launch");
    return timed_launch(MU_K_GATED_GRAD, 0.0, 0.0, s, [&] {
        hipLaunchKernelGGL(k_join, dim3((unsigned)wgs), dim3(NTHR), 0, s, j);
        return hipGetLastError();
    }, "gated feed-forward join launch");
}

template <typename T>
int run_fwd(const mu_gated* a, const Plan& p, char* ws, hipStream_t s) {
    for (const Source* q : {&p.x, &p.wg, &p.wu}) {
        const int rc = pack<T>(MU_K_GATED, *q, ws, s);
        if (rc) return rc;
    }
    TileArgs t{};
    t.a[0] = at(p.x, ws);
    t.b[0] = at(p.wg, ws);
    t.b[1] = at(p.wu, ws);
    t.lda = p.x.pitch;
    t.ldb = p.wg.pitch;
    t.m = a->tokens;
    t.n = a->hidden;
    t.k = a->dim;
    t.kt_split = 1 << 30;
    t.act = a->activation;
    t.out[0] = a->h;
    t.ldo = a->hidden;
    t.gates[0] = a->gate_out;
    t.gates[1] = a->up_out;
    const double n = (double)a->tokens, d = (double)a->dim, f = (double)a->hidden;
    return product<T, FWD>(MU_K_GATED, t, 1, 4.0 * n * d * f,
                           sizeof(T) * (n * d + 2 * d * f + (a->gate_out ? 3 : 1) * n * f), s);
}

template <typename T>
int run_bwd(const mu_gated_grad* a, const Plan& p, char* ws, hipStream_t s) {
    const double n = (double)a->tokens, d = (double)a->dim, f = (double)a->hidden;
    for (const Source* q : {&p.x, &p.wg, &p.wu}) {
        const int rc = pack<T>(MU_K_GATED_GRAD, *q, ws, s);
        if (rc) return rc;
    }
    T *dg = (T*)(ws + p.off_dg), *du = (T*)(ws + p.off_du);
    int rc = MU_OK;
    if (!a->gate) {
        TileArgs t{};
        t.a[0] = at(p.x, ws);
        t.b[0] = at(p.wg, ws);
        t.b[1] = at(p.wu, ws);
        t.lda = p.x.pitch;
        t.ldb = p.wg.pitch;
        t.m = a->tokens;
        t.n = a->hidden;
        t.k = a->dim;
        t.kt_split = 1 << 30;
        t.act = a->activation;
        t.dh = a->grad_h;
        t.out[0] = dg;
        t.out[1] = du;
        t.ldo = p.pitch_h;
        rc = product<T, RECOMP>(MU_K_GATED_GRAD, t, 1, 4.0 * n * d * f, sizeof(T) * (n * d + 2 * d * f + 3 * n * f), s);
    } else {
        rc = timed_launch(MU_K_GATED_GRAD, 0.0, 5.0 * sizeof(T) * n * f, s, [&] {
            const int64_t wgs = ceil_div(a->tokens * (p.pitch_h / vec_of<T>()), NTHR);
            hipLaunchKernelGGL(k_slopes<T>, dim3((unsigned)std::min<int64_t>(wgs, 1 << 16)), dim3(NTHR), 0, s,
                               SlopeArgs{a->grad_h, a->gate, a->up, dg, du, a->tokens, a->hidden, p.pitch_h, a->activation});
            return hipGetLastError();
        }, "gated feed-forward slopes launch");
    }
    if (rc) return rc;
    TileArgs t{};
    t.a[0] = dg;
    t.a[1] = du;
    t.lda = p.pitch_h;
    if (a->dx) {
        t.b[0] = at(p.wg, ws);
        t.b[1] = at(p.wu, ws);
        t.ldb = p.wg.pitch;
        t.m = a->tokens;
        t.n = a->dim;
        t.k = a->hidden;
        t.kt_split = p.kt_dx;
        t.out[0] = a->dx;
        t.part = p.splits_dx > 1 ? (float*)(ws + p.off_part) : nullptr;
        rc = product<T, DX>(MU_K_GATED_GRAD, t, p.splits_dx, 4.0 * n * d * f, sizeof(T) * (n * d + 2 * d * f + 2 * n * f), s);
        if (!rc && t.part) rc = join(JoinArgs{t.part, {a->dx, nullptr}, a->tokens * a->dim, p.splits_dx, 1, sizeof(T) == 4, false}, s);
        if (rc) return rc;
    }
    if (a->d_gate) {
        const bool f32 = a->grad_dtype == MU_F32;
        t.b[0] = at(p.x, ws);
        t.ldb = p.x.pitch;
        t.m = a->hidden;
        t.n = a->dim;
        t.k = a->tokens;
        t.kt_split = p.kt_dw;
        t.out[0] = a->d_gate;
        t.out[1] = a->d_up;
        t.out_f32 = f32;
        t.accumulate = a->accumulate;
        t.part = p.splits_dw > 1 ? (float*)(ws + p.off_part) : nullptr;
        rc = product<T, DW>(MU_K_GATED_GRAD, t, p.splits_dw, 4.0 * n * d * f,
                            sizeof(T) * (n * d + 2 * n * f) + es_of(a->grad_dtype) * 2 * d * f, s);
        if (!rc && t.part)
            rc = join(JoinArgs{t.part, {a->d_gate, a->d_up}, a->hidden * a->dim, p.splits_dw, 2, f32, (bool)a->accumulate}, s);
    }
    return rc;
}

struct Buf {
    const void* p;
    int64_t n;
    size_t es;
    uintptr_t lo() const { return (uintptr_t)p; }
    uintptr_t hi() const { return lo() + (size_t)n * es; }
};
bool overlap(const Buf& a, const Buf& b) { return a.p && b.p && a.n && b.n && a.lo() < b.hi() && b.lo() < a.hi(); }

template <size_t NI, size_t NO>
int check_buffers(const Buf (&in)[NI], const Buf (&out)[NO]) {
    for (const Buf& b : in)
        if (!aligned(b.p, b.es)) return fail(MU_ERR_LAYOUT, "misaligned buffer");
    for (size_t i = 0; i < NO; ++i) {
        if (!aligned(out[i].p, out[i].es)) return fail(MU_ERR_LAYOUT, "misaligned buffer");
        for (const Buf& b : in)
            if (overlap(out[i], b)) return fail(MU_ERR_LAYOUT, "an output overlaps an input");
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(MU_ERR_LAYOUT, "outputs overlap");
    }
    return MU_OK;
}

int check_sizes(int64_t tokens, int64_t dim, int64_t hidden, int dtype, int act) {
    if (dtype != MU_F32 && dtype != MU_BF16) return fail(MU_ERR_DTYPE, "unknown dtype %d", dtype);
    if (act < MU_ACT_SILU || act > MU_ACT_RELU) return fail(MU_ERR_INVALID_ARG, "unknown activation %d", act);
    if (tokens < 0 || tokens > 0x7fffffffLL) return fail(MU_ERR_INVALID_ARG, "bad token count");
    if (dim < 1 || dim > MU_GATED_MAX_DIM || hidden < 1 || hidden > MU_GATED_MAX_DIM)
        return fail(MU_ERR_INVALID_ARG, "dim and hidden must be in [1, %d]", MU_GATED_MAX_DIM);
    return MU_OK;
}

int check_fwd(const mu_gated* a) {
    if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
    int rc = check_sizes(a->tokens, a->dim, a->hidden, a->dtype, a->activation);
    if (rc) return rc;
    if (!a->gate_out != !a->up_out) return fail(MU_ERR_INVALID_ARG, "gate_out and up_out go together");
    if (a->tokens == 0) return MU_OK;
    if (!a->x || !a->w_gate || !a->w_up || !a->h) return fail(MU_ERR_INVALID_ARG, "null x, w_gate, w_up or h");
    const size_t es = es_of(a->dtype);
    const int64_t nx = a->tokens * a->dim, nw = a->hidden * a->dim, nh = a->tokens * a->hidden;
    return check_buffers({Buf{a->x, nx, es}, Buf{a->w_gate, nw, es}, Buf{a->w_up, nw, es}},
                         {Buf{a->h, nh, es}, Buf{a->gate_out, nh, es}, Buf{a->up_out, nh, es}});
}

int check_bwd(const mu_gated_grad* a) {
    if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
    int rc = check_sizes(a->tokens, a->dim, a->hidden, a->dtype, a->activation);
    if (rc) return rc;
    if (a->grad_dtype != a->dtype && a->grad_dtype != MU_F32)
        return fail(MU_ERR_DTYPE, "grad_dtype must be dtype or float32");
    if (a->accumulate != 0 && a->accumulate != 1) return fail(MU_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (!a->d_gate != !a->d_up) return fail(MU_ERR_INVALID_ARG, "d_gate and d_up go together");
    if (!a->gate != !a->up) return fail(MU_ERR_INVALID_ARG, "gate and up go together");
    if (a->tokens > 0 && (!a->grad_h || !a->x || !a->w_gate || !a->w_up))
        return fail(MU_ERR_INVALID_ARG, "null grad_h, x, w_gate or w_up");
    const size_t es = es_of(a->dtype), eg = es_of(a->grad_dtype);
    const int64_t nx = a->tokens * a->dim, nw = a->hidden * a->dim, nh = a->tokens * a->hidden;
    return check_buffers({Buf{a->grad_h, nh, es}, Buf{a->x, nx, es}, Buf{a->w_gate, nw, es}, Buf{a->w_up, nw, es},
                          Buf{a->gate, nh, es}, Buf{a->up, nh, es}},
                         {Buf{a->dx, nx, es}, Buf{a->d_gate, nw, eg}, Buf{a->d_up, nw, eg}});
}

int check_workspace(const void* ws, size_t have, size_t need) {
    if (!need) return MU_OK;
    if (!ws) return fail(MU_ERR_WORKSPACE, "workspace is null (need %zu bytes)", need);
    if (!aligned(ws, ALIGN)) return fail(MU_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (have < need) return fail(MU_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", have, need);
    return MU_OK;
}

}  // namespace

extern "C" {

int mu_gated_mlp_workspace_size(const mu_gated* a, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check_fwd(a);
        if (rc) return rc;
        *bytes = a->tokens == 0 ? 0 : plan_fwd(a).bytes;
        return MU_OK;
    });
}

int mu_gated_mlp(const mu_gated* a, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_fwd(a);
        if (rc || a->tokens == 0) return rc;
        const Plan p = plan_fwd(a);
        rc = check_workspace(ws, ws_bytes, p.bytes);
        if (rc) return rc;
        hipStream_t s = (hipStream_t)stream;
        return a->dtype == MU_BF16 ? run_fwd<bf16>(a, p, (char*)ws, s) : run_fwd<float>(a, p, (char*)ws, s);
    });
}

int mu_gated_mlp_grad_workspace_size(const mu_gated_grad* a, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check_bwd(a);
        if (rc) return rc;
        *bytes = a->tokens == 0 ? 0 : plan_bwd(a).bytes;
        return MU_OK;
    });
}

int mu_gated_mlp_grad(const mu_gated_grad* a, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_bwd(a);
        if (rc || (!a->dx && !a->d_gate)) return rc;
        hipStream_t s = (hipStream_t)stream;
        if (a->tokens == 0) {   // no rows: zero gradients
            if (!a->d_gate || a->accumulate) return MU_OK;
            return join(JoinArgs{nullptr, {a->d_gate, a->d_up}, a->hidden * a->dim, 0, 2, a->grad_dtype == MU_F32, false}, s);
        }
        const Plan p = plan_bwd(a);
        rc = check_workspace(ws, ws_bytes, p.bytes);
        if (rc) return rc;
        return a->dtype == MU_BF16 ? run_bwd<bf16>(a, p, (char*)ws, s) : run_bwd<float>(a, p, (char*)ws, s);
    });
}

}  // extern "C"
