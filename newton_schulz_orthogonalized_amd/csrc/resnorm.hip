// The norms around a block, its gate and the residual sum, with their gradients
// (gfx950): the C entry points and their kernels.
//
//   r' = a r + gate * N(y; post),  n = N(r'; pre),  N(v; w) = v s w,
//   s = (mean(v^2) + eps)^(-1/2)
//
// A team of 8 to 1024 lanes holds a row in registers between its sums: every element is
// read once and written once. Gradients, with t = dn * pre, s2 and s1 the factors
// of r' and y, D the row length:
//   d      = dr' + s2 t - s2^3 (sum t r') / D r'
//   d r    = a d
//   d pre  = sum over rows of dn * r' s2,    d gate = sum over its rows of d * N(y)
//   d post = sum over rows of d gate * y s1
//   v      = d * gate * post,  d y = s1 v - s1^3 (sum v y) / D y
// A workgroup takes a run of rows and sums their share of the three column sums
// in registers; what the workgroups leave is added up in a second launch, in
// order, so the same call gives the same bits.
//
// The gradient reads r' as the forward call stored it. With a bfloat16 residual that is
// rounded, which the sum of dn * r' shows: d pre 0.0023 of its size off (2048 x 2048) where
// an unrounded r' and the rounding of the result leave 0.0017. A float32 residual, which a
// caller may have beside bfloat16 updates, avoids it; a float32 copy of r' kept for the
// gradient alone would be three times its bytes to write and read. Everything else is
// float32 until it is stored.
//
// What bounds both: HBM (inputs cold, a large copy runs at 5.1 TB/s). Forward and gradient,
// the second launch's 4 to 7 us with it, of 8192 x 4096 bfloat16 58 and 89 us (4.7 and 4.5
// TB/s), 16384 x 2048 with a float32 residual 74 and 127 (5.4 and 4.8), 8192 x 2048 float32
// 56 and 87 (4.8 and 4.6), 262144 x 128 50 and 95 (5.4 and 4.2), 16384 x 1000 33 and 60 (4.0
// and 3.3: a third of the second run's lanes idle), 3000 x 16000 94 and 235 (4.1 and 2.5:
// registers spill, 121 MB of the 345 written), 5000 x 9001 150 and 298 (2.4 and 1.8: odd
// rows). With sums through LDS shuffles and weights read for every row the gradient of
// 8192 x 4096 took 136; holding the next row alone gained nothing there.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "../../include/muon_mi355x.h"
#include "capi_common.hpp"
#include "common.hpp"
#include "vec.hpp"

using namespace mu;

namespace {

constexpr int V = 8;   // elements of a run: one or two 16-byte accesses

// A workgroup: teams of LANES lanes (part of a wave, one, or several), a row each.
template <int LANES> constexpr int teams() { return LANES <= 64 ? 256 / LANES : 1; }
template <int LANES> constexpr int threads() { return LANES * teams<LANES>(); }

// Sums of K values over the team, in a fixed order. Alternating halves of `red`
// make one barrier a sum enough: a half is written again only behind the next
// sum's barrier.
template <int LANES, int K>
__device__ __forceinline__ void team_sums(float (&v)[K], float (*red)[K][16], int& turn) {
    wave_sums<LANES < 64 ? LANES : 64>(v);
    if constexpr (LANES > 64) {
        float(*r)[16] = red[turn];
        turn ^= 1;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) r[k][wave] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < LANES / 64; ++w) s += r[k][w];
            v[k] = s;
        }
    }
}

// A weight's run as float32, of either type; 1 where there is none.
__device__ __forceinline__ void load_weight(const void* w, bool is_bf16, int64_t at, int cnt, float (&v)[V]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 1.f;
    } else if (is_bf16) {
        load_run<bf16, V>((const bf16*)w + at, cnt, v);
    } else {
        load_run<float, V>((const float*)w + at, cnt, v);
    }
}

struct FwdArgs {
    mu_resnorm a;
    int64_t per_group;   // rows of a gate row
    float inv_dim;
};

template <typename TR, typename TY, int LANES, int NV>
__global__ __launch_bounds__(threads<LANES>()) void k_resnorm(FwdArgs A) {
    constexpr int TEAMS = teams<LANES>();
    __shared__ float red[2][1][16];
    const mu_resnorm& P = A.a;
    const int dim = (int)P.dim, lane = threadIdx.x % LANES;
    const bool wbf = P.weight_dtype == MU_BF16;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * TEAMS + threadIdx.x / LANES; row < P.rows; row += (int64_t)gridDim.x * TEAMS) {
        float r[NV][V], y[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LANES + lane) * V, cnt = dim - c;
            load_run<TR, V>((const TR*)P.residual + row * dim + c, cnt, r[j]);
            if (P.update) load_run<TY, V>((const TY*)P.update + row * dim + c, cnt, y[j]);
        }
        float f = 1.f;
        if (P.post_norm) {
            float s[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] += y[j][e] * y[j][e];
            team_sums<LANES>(s, red, turn);
            f = 1.f / sqrtf(s[0] * A.inv_dim + P.eps);
        }
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LANES + lane) * V, cnt = dim - c;
            if (P.update) {
                float w[V], g[V];
                load_weight(P.post_weight, wbf, c, cnt, w);
                load_weight(P.gate, wbf, P.gate ? row / A.per_group * dim + c : 0, cnt, g);
#pragma unroll
                for (int e = 0; e < V; ++e) r[j][e] = P.residual_scale * r[j][e] + y[j][e] * f * w[e] * g[e];
                store_run<TR, V>((TR*)P.new_residual + row * dim + c, cnt, r[j]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) r[j][e] *= P.residual_scale;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] += e < cnt ? r[j][e] * r[j][e] : 0.f;
        }
        team_sums<LANES>(s, red, turn);
        f = 1.f / sqrtf(s[0] * A.inv_dim + P.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LANES + lane) * V, cnt = dim - c;
            float w[V];
            load_weight(P.pre_weight, wbf, c, cnt, w);
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] *= r[j][e] * f;
            store_run<TY, V>((TY*)P.normed + row * dim + c, cnt, w);
        }
    }
}

struct BwdArgs {
    mu_resnorm_grad a;
    const void* r;        // r', or r where there is no update
    float r_scale;        // 1, or residual_scale
    int64_t per_group;    // rows of a gate row
    int64_t groups;
    int64_t chunk;        // rows of a workgroup within its group
    int64_t cuts;         // workgroups of a group; 1: each group's sums are finished by its workgroup
    float* pre;           // [workgroups, dim] partial sums, or null
    float* post;
    float* gate;          // [groups * cuts, dim], where cuts > 1
    float inv_dim;
};

// Add the teams' sums up and write them: as a partial row, or finished.
template <int LANES, int NV>
__device__ __forceinline__ void flush(float (&acc)[NV][V], float* part, void* out, bool out_bf16, int dim, float* lds) {
    constexpr int TEAMS = teams<LANES>();
    const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LANES + lane) * V, cnt = dim - c;
        if constexpr (TEAMS > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) lds[(team * LANES + lane) * V + e] = acc[j][e];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float s = 0.f;
#pragma unroll
                for (int t = 0; t < TEAMS; ++t) s += lds[(t * LANES + lane) * V + e];
                acc[j][e] = s;
            }
        }
        if (team == 0) {
            if (part) store_run<float, V>(part + c, cnt, acc[j]);
            else if (out_bf16) store_run<bf16, V>((bf16*)out + c, cnt, acc[j]);
            else store_run<float, V>((float*)out + c, cnt, acc[j]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) acc[j][e] = 0.f;
    }
}

template <typename TR, typename TY, int LANES, int NV>
__global__ __launch_bounds__(threads<LANES>()) void k_resnorm_grad(BwdArgs A) {
    constexpr int TEAMS = teams<LANES>();
    __shared__ float red3[2][3][16];
    __shared__ float red1[2][1][16];
    __shared__ float lds[TEAMS > 1 ? TEAMS * LANES * V : 1];
    const mu_resnorm& P = A.a.fwd;
    const int dim = (int)P.dim, lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const bool wbf = P.weight_dtype == MU_BF16;
    int turn3 = 0, turn1 = 0;
    // Column sums of rows past 4096: two of the three lie in LDS, each lane its own (two reads
    // and two writes a run beside a row's six passes over HBM); registers are short of them.
    constexpr bool IN_LDS = LANES * NV >= 1024;
    __shared__ f32x4 sums[IN_LDS ? 4 * NV * LANES : 1];
    auto kept = [&](int which, int j, int half) -> f32x4& { return sums[((which * NV + j) * 2 + half) * LANES + lane]; };
    float apre[NV][V], apost[NV][V], agate[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < V; ++e) apre[j][e] = apost[j][e] = agate[j][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 4 && IN_LDS; ++k) kept(k >> 1, j, k & 1) = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // which: 0 post, 1 gate
    auto add = [&](int which, float (&acc)[NV][V], int j, const float (&v)[V]) {
        if constexpr (IN_LDS) {
            kept(which, j, 0) += f32x4{v[0], v[1], v[2], v[3]};
            kept(which, j, 1) += f32x4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) acc[j][e] += v[e];
        }
    };
    auto fetch_sums = [&](int which, float (&acc)[NV][V]) {
        if constexpr (IN_LDS) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 x = kept(which, j, h);
                    kept(which, j, h) = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][4 * h + e] = x[e];
                }
        }
    };

    // sixteen waves have half the registers: no weights and no next row are held
    constexpr bool AHEAD = LANES < 1024;
    float wpre[NV][V], wpost[NV][V];
    auto weights = [&](int j) {
        const int c = (j * LANES + lane) * V, cnt = dim - c;
        load_weight(P.pre_weight, wbf, c, cnt, wpre[j]);
        load_weight(P.post_weight, wbf, c, cnt, wpost[j]);
    };
#pragma unroll
    for (int j = 0; j < NV && AHEAD; ++j) weights(j);
    // cuts workgroups share a group; with one each, a workgroup takes every gridDim-th group
    const int64_t step = A.cuts > 1 ? A.groups : gridDim.x;
    for (int64_t group = A.cuts > 1 ? blockIdx.x / A.cuts : blockIdx.x; group < A.groups; group += step) {
        const int64_t lo = A.cuts > 1 ? (blockIdx.x % A.cuts) * A.chunk : 0;
        const int64_t hi = min(A.per_group, lo + A.chunk);
        // a row's loads are on their way while the row before it is summed
        Run8<TR> nr[NV], nd[NV];
        Run8<TY> ny[NV], nn[NV];
        auto fetch = [&](int64_t row) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * LANES + lane) * V, cnt = dim - c;
                nr[j].load((const TR*)A.r + row * dim + c, cnt);
                if (P.update) ny[j].load((const TY*)P.update + row * dim + c, cnt);
                if (A.a.grad_residual) nd[j].load((const TR*)A.a.grad_residual + row * dim + c, cnt);
                if (A.a.grad_normed) nn[j].load((const TY*)A.a.grad_normed + row * dim + c, cnt);
            }
        };
        if (AHEAD && lo + team < hi) fetch(group * A.per_group + lo + team);
        for (int64_t i = lo + team; i < hi; i += TEAMS) {   // (TEAMS > 1 has no barrier in here)
            const int64_t row = group * A.per_group + i;
            if (!AHEAD) fetch(row);
            Run8<TR> kr[NV], kd[NV];
            Run8<TY> ky[NV], kn[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) kr[j] = nr[j], kd[j] = nd[j], ky[j] = ny[j], kn[j] = nn[j];
            if (AHEAD && i + TEAMS < hi) fetch(row + TEAMS);
            float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int cnt = dim - (j * LANES + lane) * V;
                float r[V], y[V], n[V];
                if (!AHEAD) __builtin_amdgcn_sched_barrier(0);   // one run's registers at a time
                if (!AHEAD) weights(j);
                if (A.a.grad_normed) {
                    kr[j].widen(r);
                    kn[j].widen(n);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        r[e] *= A.r_scale;
                        s[0] += r[e] * r[e];
                        s[1] += e < cnt ? n[e] * wpre[j][e] * r[e] : 0.f;
                    }
                }
                if (P.post_norm) {
                    ky[j].widen(y);
#pragma unroll
                    for (int e = 0; e < V; ++e) s[2] += y[e] * y[e];
                }
            }
            team_sums<LANES>(s, red3, turn3);
            const float f1 = P.post_norm ? 1.f / sqrtf(s[2] * A.inv_dim + P.eps) : 1.f;
            const float f2 = 1.f / sqrtf(s[0] * A.inv_dim + P.eps);
            const float c2 = f2 * (f2 * (f2 * (s[1] * A.inv_dim)));
            float d[NV][V], sv[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * LANES + lane) * V, cnt = dim - c;
                float y[V], g[V], o[V];
                if (!AHEAD) __builtin_amdgcn_sched_barrier(0);
                if (!AHEAD) weights(j);
                kd[j].widen(d[j]);
                if (!A.a.grad_residual) {
#pragma unroll
                    for (int e = 0; e < V; ++e) d[j][e] = 0.f;
                }
                if (A.a.grad_normed) {
                    float r[V], n[V];
                    kr[j].widen(r);
                    kn[j].widen(n);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float h = f2 * n[e];
                        r[e] *= A.r_scale;
                        apre[j][e] += h * r[e];
                        d[j][e] += h * wpre[j][e] - c2 * r[e];
                    }
                }
                if (A.a.d_residual) {
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = d[j][e] * P.residual_scale;
                    store_run<TR, V>((TR*)A.a.d_residual + row * dim + c, cnt, o);
                }
                if (!P.update) continue;
                load_weight(P.gate, wbf, P.gate ? group * dim + c : 0, cnt, g);
                ky[j].widen(y);
                float sg[V], sp[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float h = y[e] * f1;          // y, normed
                    sg[e] = d[j][e] * (h * wpost[j][e]);
                    d[j][e] *= g[e];
                    sp[e] = d[j][e] * h;
                    d[j][e] *= wpost[j][e];
                    sv[0] += e < cnt ? d[j][e] * y[e] : 0.f;
                }
                if (!IN_LDS || A.a.d_gate) add(1, agate, j, sg);
                if (!IN_LDS || A.post) add(0, apost, j, sp);
            }
            if (!A.a.d_update) continue;
            float c1 = 0.f;
            if (P.post_norm) {
                team_sums<LANES>(sv, red1, turn1);
                c1 = f1 * (f1 * (f1 * (sv[0] * A.inv_dim)));
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * LANES + lane) * V, cnt = dim - c;
                float y[V], o[V];
                ky[j].widen(y);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = f1 * d[j][e] - c1 * y[e];
                store_run<TY, V>((TY*)A.a.d_update + row * dim + c, cnt, o);
            }
        }
        if (A.a.d_gate) {
            fetch_sums(1, agate);
            flush<LANES, NV>(agate, A.gate ? A.gate + (int64_t)blockIdx.x * dim : nullptr,
                           (char*)A.a.d_gate + group * dim * (wbf ? 2 : 4), wbf, dim, lds);
        }
    }
    if (A.pre) flush<LANES, NV>(apre, A.pre + (int64_t)blockIdx.x * dim, nullptr, false, dim, lds);
    fetch_sums(0, apost);
    if (A.post) flush<LANES, NV>(apost, A.post + (int64_t)blockIdx.x * dim, nullptr, false, dim, lds);
}

// Column sums of partial rows, in order: a workgroup sums 64 columns of one
// output row, each of its 16 waves a run of the partial rows.
struct ColArgs {
    const float* part[3];   // pre, post, gate
    void* out[3];           // null: none
    int64_t rows[3];        // partial rows of an output row
    int64_t groups;         // output rows of the gate
    int dim;
    bool out_bf16;
};
constexpr int COL_WAVES = 16;

__global__ __launch_bounds__(64 * COL_WAVES) void k_colsum(ColArgs A) {
    __shared__ float part[COL_WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    const int64_t y = blockIdx.y;   // pre, post, then the gate's rows
    const int kind = y < 2 ? (int)y : 2;
    if (!A.out[kind]) return;
    const int64_t n = A.rows[kind], per = (n + COL_WAVES - 1) / COL_WAVES, group = kind == 2 ? y - 2 : 0;
    const MU_GLOBAL float* p = gp(A.part[kind]) + group * n * A.dim + c;
    float s = 0.f;
    if (c < A.dim) {
        int64_t i = wave * per;
        const int64_t end = min(n, i + per);
        for (; i + 8 <= end; i += 8) {   // eight on their way at a time
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = p[(i + k) * A.dim];
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
        for (; i < end; ++i) s += p[i * A.dim];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= A.dim) return;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < COL_WAVES; ++w) s += part[w][lane];
    const int64_t at = group * A.dim + c;
    if (A.out_bf16) ((MU_GLOBAL bf16*)A.out[kind])[at] = (bf16)s;
    else ((MU_GLOBAL float*)A.out[kind])[at] = s;
}

size_t es_of(int dtype) { return dtype == MU_BF16 ? 2 : 4; }

bool known(int dtype) { return dtype == MU_F32 || dtype == MU_BF16; }

struct Buf {
    const void* p;
    int64_t n;
    size_t es;
    uintptr_t lo() const { return (uintptr_t)p; }
    uintptr_t hi() const { return lo() + (size_t)n * es; }
};
bool overlap(const Buf& a, const Buf& b) { return a.p && b.p && a.n && b.n && a.lo() < b.hi() && b.lo() < a.hi(); }

int check_common(const mu_resnorm* a) {
    if (!known(a->residual_dtype) || !known(a->dtype) || !known(a->weight_dtype)) return fail(MU_ERR_DTYPE, "unknown dtype");
    if (a->residual_dtype == MU_BF16 && a->dtype == MU_F32)
        return fail(MU_ERR_DTYPE, "a bfloat16 residual takes no float32 update");
    if (a->dim < 1 || a->dim > MU_RESNORM_MAX_DIM) return fail(MU_ERR_INVALID_ARG, "dim must be in [1, %d]", MU_RESNORM_MAX_DIM);
    if (a->rows < 0 || a->rows > ((int64_t)1 << 40)) return fail(MU_ERR_INVALID_ARG, "bad row count");
    if (a->groups < (a->rows > 0 ? 1 : 0) || (a->rows > 0 && a->rows % a->groups != 0) || a->groups > ((int64_t)1 << 40))
        return fail(MU_ERR_INVALID_ARG, "groups must be >= 1 (no rows: >= 0) and divide rows");
    if (a->post_norm != 0 && a->post_norm != 1) return fail(MU_ERR_INVALID_ARG, "post_norm must be 0 or 1");
    if (!std::isfinite(a->residual_scale)) return fail(MU_ERR_INVALID_ARG, "residual_scale must be finite");
    if (!(a->eps > 0.f) || !std::isfinite(a->eps)) return fail(MU_ERR_INVALID_ARG, "eps must be > 0 and finite");
    if (a->post_weight && !a->post_norm) return fail(MU_ERR_INVALID_ARG, "post_weight without post_norm");
    if (!a->gate && a->groups > 1) return fail(MU_ERR_INVALID_ARG, "groups without a gate");
    return MU_OK;
}

// Lanes of a row and runs of a lane. Short rows share a wave: 510012 rows of 64 with a wave
// each took 1.1 ms both ways. The gradient's rows are four runs, the next row's four and
// three sums: two runs a lane fill the registers of eight waves, and sixteen waves have half
// as many, so past 8192 it keeps no row ahead.
template <template <typename, typename, int, int> class L, typename TR, typename TY, bool GRAD, typename... X>
hipError_t by_dim(int64_t dim, X&&... x) {
    if (dim <= 64) return L<TR, TY, 8, 1>::go(x...);
    if (dim <= 128) return L<TR, TY, 16, 1>::go(x...);
    if (dim <= 256) return L<TR, TY, 32, 1>::go(x...);
    if (dim <= 512) return L<TR, TY, 64, 1>::go(x...);
    if (dim <= 1024) return L<TR, TY, 64, 2>::go(x...);
    if (dim <= 2048) return L<TR, TY, 256, 1>::go(x...);
    if constexpr (GRAD) {
        if (dim <= 4096) return L<TR, TY, 512, 1>::go(x...);
        if (dim <= 8192) return L<TR, TY, 512, 2>::go(x...);
    } else {
        if (dim <= 4096) return L<TR, TY, 256, 2>::go(x...);
        if (dim <= 8192) return L<TR, TY, 1024, 1>::go(x...);
    }
    return L<TR, TY, 1024, 2>::go(x...);
}
template <template <typename, typename, int, int> class L, bool GRAD, typename... X>
hipError_t by_type(const mu_resnorm& a, X&&... x) {
    if (a.dtype == MU_F32) return by_dim<L, float, float, GRAD>(a.dim, x...);
    if (a.residual_dtype == MU_F32) return by_dim<L, float, bf16, GRAD>(a.dim, x...);
    return by_dim<L, bf16, bf16, GRAD>(a.dim, x...);
}

template <typename TR, typename TY, int LANES, int NV>
struct Fwd {
    static hipError_t go(const FwdArgs& f, hipStream_t s) {
        const int64_t teams_needed = (f.a.rows + teams<LANES>() - 1) / teams<LANES>();
        const unsigned grid = (unsigned)std::min<int64_t>(teams_needed, 1 << 20);
        hipLaunchKernelGGL((k_resnorm<TR, TY, LANES, NV>), dim3(grid), dim3(threads<LANES>()), 0, s, f);
        return hipGetLastError();
    }
};
template <typename TR, typename TY, int LANES, int NV>
struct Bwd {
    static hipError_t go(const BwdArgs& b, unsigned grid, hipStream_t s) {
        hipLaunchKernelGGL((k_resnorm_grad<TR, TY, LANES, NV>), dim3(grid), dim3(threads<LANES>()), 0, s, b);
        return hipGetLastError();
    }
};

// Workgroups of a gradient call and what they leave for the second launch.
struct GradPlan {
    int64_t chunk, cuts, grid;
    bool part_gate;
    size_t off_pre, off_post, off_gate, bytes;
};
constexpr int TARGET_WGS = 512;   // two workgroups of four waves a compute unit, one of eight
constexpr int MIN_ROWS = 4;       // rows of a workgroup at least: its partial sums are three rows

GradPlan plan_of(const mu_resnorm_grad* a) {
    const mu_resnorm& f = a->fwd;
    GradPlan p{};
    const int64_t per_group = f.rows ? f.rows / f.groups : 0, target = f.dim > 2048 ? TARGET_WGS / 2 : TARGET_WGS;
    const int64_t least = f.dim <= 64 ? 32 : f.dim <= 128 ? 16 : f.dim <= 256 ? 8 : MIN_ROWS;   // a row for each team
    p.cuts = std::max<int64_t>(1, std::min(target / std::max<int64_t>(1, f.groups), (per_group + least - 1) / least));
    p.chunk = per_group > 0 ? (per_group + p.cuts - 1) / p.cuts : 1;
    if (per_group > 0) p.cuts = (per_group + p.chunk - 1) / p.chunk;
    p.grid = f.rows == 0 ? 0 : p.cuts > 1 ? f.groups * p.cuts : std::min(f.groups, target);
    p.part_gate = a->d_gate && (p.cuts > 1 || f.rows == 0);
    auto take = [&](bool wanted, int64_t rows) {
        const size_t at = p.bytes;
        if (wanted) p.bytes += align_up(sizeof(float) * (size_t)rows * (size_t)f.dim);
        return at;
    };
    p.off_pre = take(a->d_pre, p.grid);
    p.off_post = take(a->d_post, p.grid);
    p.off_gate = take(p.part_gate, p.grid);
    return p;
}

int check_grad(const mu_resnorm_grad* a) {
    if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
    const mu_resnorm& f = a->fwd;
    int rc = check_common(&f);
    if (rc) return rc;
    if (a->d_gate && !f.gate) return fail(MU_ERR_INVALID_ARG, "d_gate without a gate");
    if (a->d_post && !f.post_weight) return fail(MU_ERR_INVALID_ARG, "d_post without post_weight");
    if (a->d_pre && !f.pre_weight) return fail(MU_ERR_INVALID_ARG, "d_pre without pre_weight");
    if (!f.update && f.rows > 0 && (f.gate || f.post_norm || a->d_update))
        return fail(MU_ERR_INVALID_ARG, "gate, post_norm or d_update without update");
    if (!f.update && a->grad_residual) return fail(MU_ERR_INVALID_ARG, "grad_residual without update");
    if (f.groups > 60000 && f.rows == 0) return fail(MU_ERR_INVALID_ARG, "too many groups for no rows");
    const void* r = f.update ? f.new_residual : f.residual;
    if (f.rows > 0 && !r) return fail(MU_ERR_INVALID_ARG, "new_residual (residual without update) is null");
    const size_t er = es_of(f.residual_dtype), ey = es_of(f.dtype), ew = es_of(f.weight_dtype);
    const int64_t n = f.rows * f.dim;
    const Buf in[] = {{r, n, er}, {f.update, n, ey}, {f.gate, f.groups * f.dim, ew}, {f.post_weight, f.dim, ew},
                      {f.pre_weight, f.dim, ew}, {a->grad_residual, n, er}, {a->grad_normed, n, ey}};
    const Buf out[] = {{a->d_residual, n, er}, {a->d_update, n, ey}, {a->d_gate, f.groups * f.dim, ew},
                       {a->d_post, f.dim, ew}, {a->d_pre, f.dim, ew}};
    for (const Buf& b : in)
        if (!aligned(b.p, b.es)) return fail(MU_ERR_LAYOUT, "misaligned buffer");
    for (size_t i = 0; i < 5; ++i) {
        if (!aligned(out[i].p, out[i].es)) return fail(MU_ERR_LAYOUT, "misaligned buffer");
        for (const Buf& b : in)
            if (overlap(out[i], b)) return fail(MU_ERR_LAYOUT, "a gradient overlaps an input");
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(MU_ERR_LAYOUT, "gradients overlap");
    }
    return MU_OK;
}

}  // namespace

extern "C" {

int mu_residual_norm(const mu_resnorm* a, void* stream) {
    return guarded([&]() -> int {
        if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
        int rc = check_common(a);
        if (rc) return rc;
        if (a->rows == 0) return MU_OK;
        if (!a->update && (a->new_residual || a->gate || a->post_norm))
            return fail(MU_ERR_INVALID_ARG, "new_residual, gate or post_norm without update");
        if (!a->residual || !a->normed || (a->update && !a->new_residual))
            return fail(MU_ERR_INVALID_ARG, "null residual, new_residual or normed");
        const size_t er = es_of(a->residual_dtype), ey = es_of(a->dtype), ew = es_of(a->weight_dtype);
        const int64_t n = a->rows * a->dim;
        const Buf in[] = {{a->residual, n, er}, {a->update, n, ey}, {a->gate, a->groups * a->dim, ew},
                          {a->post_weight, a->dim, ew}, {a->pre_weight, a->dim, ew}};
        const Buf out[] = {{a->new_residual, n, er}, {a->normed, n, ey}};
        for (const Buf& b : in)
            if (!aligned(b.p, b.es)) return fail(MU_ERR_LAYOUT, "misaligned buffer");
        for (int i = 0; i < 2; ++i) {
            if (!aligned(out[i].p, out[i].es)) return fail(MU_ERR_LAYOUT, "misaligned buffer");
            for (const Buf& b : in) {
                // in place: every element is read before it is written
                const bool same = out[i].p == b.p && out[i].es == b.es && (&b == &in[0] || &b == &in[1]);
                if (overlap(out[i], b) && !same) return fail(MU_ERR_LAYOUT, "an output overlaps an input");
            }
        }
        if (overlap(out[0], out[1])) return fail(MU_ERR_LAYOUT, "outputs overlap");
        FwdArgs f{*a, a->rows / a->groups, 1.f / (float)a->dim};
        hipStream_t s = (hipStream_t)stream;
        const double bytes = (double)n * (a->update ? 2.0 * er + 2.0 * ey : (double)(er + ey));
        return timed_launch(MU_K_RESNORM, 9.0 * (double)n, bytes, s, [&] { return by_type<Fwd, false>(*a, f, s); },
                            "residual norm launch");
    });
}

int mu_residual_norm_grad_workspace_size(const mu_resnorm_grad* a, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check_grad(a);
        if (rc) return rc;
        *bytes = plan_of(a).bytes;
        return MU_OK;
    });
}

int mu_residual_norm_grad(const mu_resnorm_grad* a, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_grad(a);
        if (rc) return rc;
        const mu_resnorm& f = a->fwd;
        const GradPlan p = plan_of(a);
        if (p.bytes) {
            if (!ws) return fail(MU_ERR_WORKSPACE, "workspace is null (need %zu bytes)", p.bytes);
            if (!aligned(ws, ALIGN)) return fail(MU_ERR_WORKSPACE, "workspace must be 256-byte aligned");
            if (ws_bytes < p.bytes) return fail(MU_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, p.bytes);
        }
        char* w = (char*)ws;
        BwdArgs b{};
        b.a = *a;
        b.r = f.update ? f.new_residual : f.residual;
        b.r_scale = f.update ? 1.f : f.residual_scale;
        b.per_group = f.rows ? f.rows / f.groups : 0;
        b.groups = f.groups;
        b.chunk = p.chunk;
        b.cuts = p.cuts;
        b.pre = a->d_pre ? (float*)(w + p.off_pre) : nullptr;
        b.post = a->d_post ? (float*)(w + p.off_post) : nullptr;
        b.gate = p.part_gate ? (float*)(w + p.off_gate) : nullptr;
        b.inv_dim = 1.f / (float)f.dim;
        hipStream_t s = (hipStream_t)stream;
        const double n = (double)f.rows * (double)f.dim, er = (double)es_of(f.residual_dtype), ey = (double)es_of(f.dtype);
        const double bytes = n * (er + (f.update ? ey : 0) + (a->grad_residual ? er : 0) + (a->grad_normed ? ey : 0) +
                                  (a->d_residual ? er : 0) + (a->d_update ? ey : 0));
        if (p.grid > 0) {
            rc = timed_launch(MU_K_RESNORM_GRAD, 17.0 * n, bytes, s,
                              [&] { return by_type<Bwd, true>(f, b, (unsigned)p.grid, s); }, "residual norm gradient launch");
            if (rc) return rc;
        }
        if (!a->d_pre && !a->d_post && !p.part_gate) return MU_OK;
        ColArgs c{{b.pre, b.post, b.gate}, {a->d_pre, a->d_post, p.part_gate ? a->d_gate : nullptr},
                  {p.grid, p.grid, f.rows == 0 ? 0 : p.cuts}, f.groups, (int)f.dim, f.weight_dtype == MU_BF16};
        return timed_launch(MU_K_RESNORM_GRAD, 0.0, 0.0, s, [&] {
            const dim3 grid((unsigned)((f.dim + 63) / 64), (unsigned)(2 + (p.part_gate ? f.groups : 0)));
            hipLaunchKernelGGL(k_colsum, grid, dim3(64 * COL_WAVES), 0, s, c);
            return hipGetLastError();
        }, "residual norm gradient sums launch");
    });
}

}  // extern "C"
