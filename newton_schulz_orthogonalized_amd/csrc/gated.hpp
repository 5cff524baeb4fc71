// Shared by the sources of the gated feed-forward block: activations, the tiled
// products' arguments, operand addressing and the order of tiles.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/muon_mi355x.h"
#include "common.hpp"
#include "vec.hpp"

namespace mu {
namespace gated {

constexpr int NTHR = 256;
#define LDSP __attribute__((address_space(3)))
constexpr int BUF_RAW32 = 0x00020000;   // word 3 of a raw buffer resource
constexpr int OUTSIDE = 0x7fffff00;     // an offset beyond every resource: reads zeros

enum Mode : int { FWD, RECOMP, DX, DW };

template <int N>
struct Stage {
    static constexpr int value = N;
};
// fn(Stage<i>{}) for i = B .. E-1, every index a compile-time constant
template <int B, int E, typename Fn>
__device__ __forceinline__ void static_for(Fn&& fn) {
    if constexpr (B < E) {
        fn(Stage<B>{});
        static_for<B + 1, E>(fn);
    }
}

// ---------------------------------------------------------------------------
// Activations: act(g) and its derivative, float32
// ---------------------------------------------------------------------------
// 1 / (1 + e^-z); the exponential's overflow gives 0. FAST: the hardware's
// exponential and reciprocal (each within 2^-22), where results become bfloat16.
template <bool FAST>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + __expf(-z));
    else return 1.f / (1.f + expf(-z));
}
template <bool FAST>
__device__ __forceinline__ void act_of(int kind, float g, float& a, float& slope) {
    switch (kind) {
        case MU_ACT_SILU: {
            const float s = sigmoid<FAST>(g);
            a = g * s;
            slope = s * (1.f + g * (1.f - s));
            return;
        }
        case MU_ACT_GELU: {   // g Phi(g); slope Phi(g) + g phi(g)
            float c, e;
            if constexpr (FAST) {
                // Phi(-x sqrt(2)) = erfc(x) / 2 = e^(-x^2) t P(t) / 2, t = 1 / (1 + 0.45 x): P is
                // a least-squares fit to erfc(x) e^(x^2) / t at Chebyshev points of x in [0, 14],
                // 5e-7 of it at most (the library's erfc took 11 us more for a 256 x 256 tile)
                e = __expf(-0.5f * g * g);
                const float t = __builtin_amdgcn_rcpf(1.f + 0.45f * 0.70710678f * fabsf(g));
                float p = 0.06890473f;
                p = p * t - 0.24888976f;
                p = p * t + 0.22391099f;
                p = p * t + 0.02623324f;
                p = p * t + 0.196169f;
                p = p * t + 0.22578287f;
                p = p * t + 0.2540041f;
                p = p * t + 0.25388519f;
                c = 0.5f * e * t * p;
                c = g < 0.f ? c : 1.f - c;
            } else {
                c = 0.5f * erfcf(g * -0.70710678f);
                e = expf(-0.5f * g * g);
            }
            a = g * c;
            slope = c + g * 0.39894228f * e;
            return;
        }
        case MU_ACT_GELU_TANH: {   // g (1 + tanh z) / 2 = g sigmoid(2 z)
            const float k = 0.79788456f, q = 0.044715f;
            const float s = sigmoid<FAST>(2.f * k * (g + q * g * g * g));
            a = g * s;
            // (far from zero s is 1 or 0, and the factor's square may have left float32)
            const float t = g * s * (1.f - s);
            slope = t == 0.f ? s : s + t * (2.f * k * (1.f + 3.f * q * g * g));
            return;
        }
        default:
            a = fmaxf(g, 0.f);
            slope = g > 0.f ? 1.f : 0.f;
            if (g != g) a = g;
    }
}

// act(g), and with its slope, of a run; the kind is decided once for all of it.
template <bool FAST, int V>
__device__ __forceinline__ void act_run(int kind, const float (&g)[V], float (&a)[V]) {
    float s;
#define MU_RUN(K)                                    \
    case K:                                          \
        _Pragma("unroll") for (int e = 0; e < V; ++e) act_of<FAST>(K, g[e], a[e], s); \
        return;
    switch (kind) { MU_RUN(MU_ACT_SILU) MU_RUN(MU_ACT_GELU) MU_RUN(MU_ACT_GELU_TANH) MU_RUN(MU_ACT_RELU) }
#undef MU_RUN
}
template <bool FAST, int V>
__device__ __forceinline__ void slope_run(int kind, const float (&g)[V], float (&a)[V], float (&s)[V]) {
#define MU_RUN(K)                                    \
    case K:                                          \
        _Pragma("unroll") for (int e = 0; e < V; ++e) act_of<FAST>(K, g[e], a[e], s[e]); \
        return;
    switch (kind) { MU_RUN(MU_ACT_SILU) MU_RUN(MU_ACT_GELU) MU_RUN(MU_ACT_GELU_TANH) MU_RUN(MU_ACT_RELU) }
#undef MU_RUN
}

// ---------------------------------------------------------------------------
// The tiled product
// ---------------------------------------------------------------------------
struct TileArgs {
    const void* a[2];
    const void* b[2];
    int64_t lda, ldb;          // row pitches in elements
    int64_t m, n, k;           // rows, columns (FWD: of h), and k (DX: of each half)
    int tiles_m, tiles_n;
    int kt_split;              // k slices of a split (blockIdx.y)
    int act;
    void* out[2];              // FWD: h; RECOMP: dg, du; DX: dx; DW: dWg, dWu
    int64_t ldo;
    void* gates[2];            // FWD: g and u, or null
    const void* dh;            // RECOMP
    float* part;               // DX, split: [splits][m][n] float32 sums
    bool out_f32;              // DW: float32 results
    bool gates_f32;            // FWD: g and u leave as float32, unrounded
    bool accumulate;           // DW
    bool aligned;              // the wide kernel: results' rows start at 16-byte steps
};

// The 256 x 256 kernel (bfloat16): one workgroup a compute unit, which takes tile
// after tile.
hipError_t launch_wide(int mode, const TileArgs& a, int grid, hipStream_t s);

template <typename T> constexpr int bk() { return 128 / (int)sizeof(T); }

template <typename T> struct Mma;
template <> struct Mma<bf16> {
    typedef bf16x8 Frag;   // k 8 (l >> 4) .. of row l & 15; two of them cover a slice
};
template <> struct Mma<float> {
    typedef f32x4 Frag;    // k 4 (l >> 4) .. of row l & 15: one of each goes to each of four instructions
};

__device__ __forceinline__ f32x4 mma(const bf16x8& a, const bf16x8& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const f32x4& a, const f32x4& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

// A resource of `bytes` from p on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const char* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, BUF_RAW32);
}

// Swizzle of the 16-byte chunks of LDS row k of an operand with k down its rows (of
// `rowb` bytes): the four rows (of both types' reads) that one access touches, and for
// bfloat16 those of the neighbouring lane group, fall into different banks.
template <typename T>
__device__ __forceinline__ int swz_down(int k, int rowb) {
    if (sizeof(T) == 4) return 4 * ((k >> 2) & 3);
    return rowb == 128 ? (k & 2) | ((k >> 1) & 4) : 2 * ((k & 3) | ((k >> 1) & 4));
}

template <typename T, int TS, bool DOWN>
struct Operand {
    static constexpr int ES = sizeof(T), NI = TS / 32;        // direct loads of a wave and slice
    static constexpr int ROWB = DOWN ? TS * ES : 128;         // bytes of an LDS row
    static constexpr int RPB = 1024 / ROWB, LPR = 64 / RPB;   // LDS rows of a load, lanes of a row

    // Load instruction i: LDS row and global 16-byte chunk of this lane.
    __device__ static __forceinline__ int lds_row(int i, int wave, int lane) { return (i * 4 + wave) * RPB + lane / LPR; }
    __device__ static __forceinline__ int chunk(int row, int lane) {
        const int p = lane % LPR;
        return DOWN ? p ^ swz_down<T>(row, ROWB) : p ^ (row & 7);
    }
    // This lane's offsets in the reads of a slice's fragments from row or column `base` on:
    // for each k half of rows, or for each 16 columns (DOWN). Opaque, so that each address is
    // an array, one of these and a constant: the compiler's alias analysis follows an address
    // over a few steps only, and where it loses it a read waits for every load on its way.
    __device__ static __forceinline__ void offsets(int (&o)[4], int base, int lane) {
        const int i = lane & 15, g = lane >> 4;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if constexpr (!DOWN) {
                o[n] = (base + i) * 128 + ((((n & 1) * 4 + g) ^ (i & 7)) << 4);
            } else if constexpr (ES == 2) {
                // lane i of each 16-lane group addresses 4 elements of row i / 4 and
                // receives column i of those four rows (see ds_read_b64_tr_b16)
                const int r = 8 * g + (i >> 2);
                o[n] = r * ROWB + ((((base + n * 16) >> 3) + ((i >> 1) & 1)) ^ swz_down<T>(r, ROWB)) * 16 + 8 * (i & 1);
            } else {
                const int col = base + n * 16 + i;
                o[n] = 4 * g * ROWB + ((col >> 2) ^ swz_down<T>(4 * g, ROWB)) * 16 + (col & 3) * 4;
            }
            asm("" : "+v"(o[n]));
        }
    }
    // Fragment f (16 rows or columns) of part kk of a slice.
    __device__ static __forceinline__ typename Mma<T>::Frag read(const char* lds, const int (&o)[4], int f, int kk) {
        if constexpr (!DOWN) {
            return *(const typename Mma<T>::Frag*)(lds + o[kk] + f * 2048);
        } else if constexpr (ES == 2) {
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDSP i16x4*)(lds + o[f] + kk * 32 * ROWB));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDSP i16x4*)(lds + o[f] + (kk * 32 + 4) * ROWB));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *(const float*)(lds + o[f] + (kk * 16 + i) * ROWB);
            return v;
        }
    }
};

// Tiles in groups of eight rows, column by column inside a group: workgroups that
// run together share eight strips of one operand and a few of the other.
__device__ __forceinline__ void tile_of(int t, int tm, int tn, int& ti, int& tj) {
    constexpr int G = 8;
    const int per = G * tn, g = t / per, w = t - g * per, gm = min(G, tm - g * G);
    ti = g * G + w % gm;
    tj = w / gm;
}

}  // namespace gated
}  // namespace mu
