// Runs of up to V elements at any element address, as float32 in registers.
// gfx950 takes global vector accesses at any address, so a whole run is one or
// two 16-byte accesses wherever it lies; a cut one goes element by element.
#pragma once

#include "common.hpp"

namespace mu {

typedef bf16x8 bf16x8u __attribute__((aligned(2)));
typedef f32x4 f32x4u __attribute__((aligned(4)));

// Elements of one 16-byte access.
template <typename T> constexpr int vec_of() { return 16 / (int)sizeof(T); }

template <typename T> struct VecOf;
template <> struct VecOf<bf16> { typedef bf16x8 V; typedef bf16x8u U; };
template <> struct VecOf<float> { typedef f32x4 V; typedef f32x4u U; };

// One 16-byte vector of up to W elements, as stored; zeros behind cnt.
template <typename T>
__device__ __forceinline__ typename VecOf<T>::V load_vec(const T* q, int cnt) {
    constexpr int W = vec_of<T>();
    const MU_GLOBAL T* p = gp(q);
    if (cnt >= W) return *(const MU_GLOBAL typename VecOf<T>::U*)p;
    typename VecOf<T>::V x;
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = e < cnt ? p[e] : (T)0.f;
    return x;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* q, int cnt, const typename VecOf<T>::V& x) {
    constexpr int W = vec_of<T>();
    MU_GLOBAL T* p = gp(q);
    if (cnt >= W) {
        *(MU_GLOBAL typename VecOf<T>::U*)p = x;
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < cnt) p[e] = x[e];
    }
}

// Eight elements of up to cnt that exist, as stored, to be widened later.
template <typename T>
struct Run8 {
    static constexpr int W = vec_of<T>(), N = 8 / W;
    typename VecOf<T>::V x[N];
    __device__ __forceinline__ void load(const T* p, int cnt) {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = load_vec<T>(p + j * W, cnt - j * W);
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f32<T>(x[e / W][e % W]);
    }
};

// v[e] = p[e] for e < cnt, 0 behind them. V is a multiple of the type's vector.
template <typename T, int V>
__device__ __forceinline__ void load_run(const T* q, int cnt, float (&v)[V]) {
    constexpr int W = vec_of<T>();
    static_assert(V % W == 0, "whole vectors");
    const MU_GLOBAL T* p = gp(q);
    if (cnt >= V) {
#pragma unroll
        for (int j = 0; j < V / W; ++j) {
            const typename VecOf<T>::V x = *(const MU_GLOBAL typename VecOf<T>::U*)(p + j * W);
#pragma unroll
            for (int e = 0; e < W; ++e) v[j * W + e] = to_f32<T>(x[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = e < cnt ? to_f32<T>(p[e]) : 0.f;
    }
}

// p[e] = v[e] for e < cnt, rounded to nearest even.
template <typename T, int V>
__device__ __forceinline__ void store_run(T* q, int cnt, const float (&v)[V]) {
    constexpr int W = vec_of<T>();
    static_assert(V % W == 0, "whole vectors");
    MU_GLOBAL T* p = gp(q);
    if (cnt >= V) {
#pragma unroll
        for (int j = 0; j < V / W; ++j) {
            typename VecOf<T>::V x;
#pragma unroll
            for (int e = 0; e < W; ++e) x[e] = from_f32<T>(v[j * W + e]);
            *(MU_GLOBAL typename VecOf<T>::U*)(p + j * W) = x;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < cnt) p[e] = from_f32<T>(v[e]);
    }
}

// Sums of K values over each run of N lanes (8 to 64) in a fixed order, in every lane: pairs,
// quads, halves of a row of 16 lanes, rows, then rows of 16 and of 32 swapped. All in vector
// instructions: with these in the place of shuffles through LDS, and weights held in
// registers, the norms' gradient of 8192 x 4096 went from 136 to 93 us.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int N, int K>
__device__ __forceinline__ void wave_sums(float (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = dpp_add<0xb1>(v[k]);    // quad_perm 1 0 3 2
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = dpp_add<0x4e>(v[k]);    // quad_perm 2 3 0 1
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = dpp_add<0x141>(v[k]);   // row_half_mirror
#pragma unroll
    for (int k = 0; k < K && N >= 16; ++k) v[k] = dpp_add<0x140>(v[k]);   // row_mirror
#pragma unroll
    for (int k = 0; k < K && N >= 32; ++k) {
        const unsigned u = __builtin_bit_cast(unsigned, v[k]);
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        v[k] = __builtin_bit_cast(float, (unsigned)p[0]) + __builtin_bit_cast(float, (unsigned)p[1]);
    }
#pragma unroll
    for (int k = 0; k < K && N == 64; ++k) {
        const unsigned u = __builtin_bit_cast(unsigned, v[k]);
        const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        v[k] = __builtin_bit_cast(float, (unsigned)p[0]) + __builtin_bit_cast(float, (unsigned)p[1]);
    }
}

}  // namespace mu
