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

}  // namespace mu
