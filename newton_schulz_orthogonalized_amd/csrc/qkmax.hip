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

#define LDSP __attribute__((address_space(3)))
// s_waitcnt with vmcnt(n) and lgkmcnt(0) (gfx9 encoding)
#define MU_WAIT_VMCNT_LGKM0(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (0 << 8) | (((n) >> 4) << 14))
constexpr int BUF_RAW32 = 0x00020000;   // word 3 of a raw buffer resource

typedef float f32x16 __attribute__((ext_vector_type(16)));

// A unit of work is a tile of BM queries of one head against at most KC keys of
// its sequence. The units of one query head are the same for every head: the
// plan kernel writes them as records, sequence by sequence, key chunk by key
// chunk (chunk c is seen by the query tiles t >= tmin(c)).
struct Unit {
    int64_t q_off, k_off;   // elements before its first query and key row (without the head)
    int32_t rows, keys;     // of this unit, both >= 1
    int32_t see;            // row i sees the unit's keys j < see + i (all of them where not causal)
    int32_t pad;
};
struct QkMaxArgs {
    mu_qk_logits p;
    const int64_t* count;    // units of one head
    const Unit* units;
    int64_t key_chunk;       // KC, a multiple of the key tile
};

struct Seq {
    int64_t q0, k0;   // element offset of its first row (without the head)
    int64_t nq, nk;
};

__device__ inline int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

__device__ inline Seq seq_of(const mu_qk_logits& A, int64_t b) {
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

// First query tile that sees key chunk c: its last row sees key c * KC.
__device__ inline int64_t tile_min(const Seq& S, int causal, int64_t kc, int bm, int64_t c) {
    const int64_t x = c * kc - (S.nk - S.nq);
    return causal && x > 0 ? x / bm : 0;
}

__device__ inline int64_t units_of(const Seq& S, int causal, int64_t kc, int bm) {
    if (S.nq <= 0 || S.nk <= 0) return 0;
    const int64_t tq = (S.nq + bm - 1) / bm, nc = (S.nk + kc - 1) / kc;
    int64_t n = 0;
    for (int64_t c = 0; c < nc; ++c) n += tq - tile_min(S, causal, kc, bm, c);
    return n;
}

// The units of chunk c of a sequence that follow record `at`, every `step`-th from `first` on.
__device__ inline void put_units(const Seq& S, const QkMaxArgs& A, int bm, int64_t c, Unit* at, int first, int step) {
    const int64_t kc = A.key_chunk, tq = (S.nq + bm - 1) / bm, t0 = tile_min(S, A.p.causal, kc, bm, c);
    const int64_t off = S.nk - S.nq, k_lo = c * kc;
    for (int64_t t = t0 + first; t < tq; t += step) {
        Unit u;
        u.q_off = S.q0 + t * bm * A.p.q_stride_s;
        u.k_off = S.k0 + k_lo * A.p.k_stride_s;
        u.rows = (int32_t)min<int64_t>(bm, S.nq - t * bm);
        const int64_t k_hi = A.p.causal ? min<int64_t>(S.nk, t * bm + u.rows + off) : S.nk;
        u.keys = (int32_t)min<int64_t>(kc, k_hi - k_lo);
        // beyond the keys on one side and below the first row's reach on the other any value does
        u.see = A.p.causal ? (int32_t)clamp64(t * bm + 1 + off - k_lo, -bm, u.keys) : u.keys;
        u.pad = 0;
        at[t - t0] = u;
    }
}

// One workgroup: the units of every sequence, and zeros to take maxima from.
// Sequences of few units are written by a thread each, others by a wave.
constexpr int PLAN_THR = 1024, PLAN_FEW = 4;
__global__ __launch_bounds__(PLAN_THR) void k_qk_plan(QkMaxArgs A, int64_t* count, Unit* units, int bm) {
    __shared__ int64_t wsum[PLAN_THR / 64], base[PLAN_THR];
    __shared__ int many;
    const int tid = threadIdx.x, wave = tid >> 6;
    if (!A.p.accumulate)
        for (int i = tid; i < A.p.q_heads; i += PLAN_THR) gp(A.p.max_logit)[i] = 0.f;
    int64_t carry = 0;
    for (int64_t b0 = 0; b0 < A.p.batch; b0 += PLAN_THR) {
        const int64_t b = b0 + tid;
        Seq S{0, 0, 0, 0};
        if (b < A.p.batch) S = seq_of(A.p, b);
        const int64_t mine = units_of(S, A.p.causal, A.key_chunk, bm);
        if (tid == 0) many = 0;
        int64_t n = mine;
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t up = __shfl_up(n, off, 64);
            if ((tid & 63) >= off) n += up;
        }
        if ((tid & 63) == 63) wsum[wave] = n;
        __syncthreads();
        int64_t before = carry + n - mine;
        for (int w = 0; w < PLAN_THR / 64; ++w) {
            if (w < wave) before += wsum[w];
            carry += wsum[w];
        }
        base[tid] = mine > PLAN_FEW ? before : -1;
        if (mine > PLAN_FEW) many = 1;
        else
            for (int64_t c = 0, at = before; at < before + mine; ++c) {
                put_units(S, A, bm, c, units + at, 0, 1);
                at += (S.nq + bm - 1) / bm - tile_min(S, A.p.causal, A.key_chunk, bm, c);
            }
        __syncthreads();
        if (many)
            for (int i = wave; i < PLAN_THR && b0 + i < A.p.batch; i += PLAN_THR / 64) {
                int64_t at = base[i];
                if (at < 0) continue;
                const Seq T = seq_of(A.p, b0 + i);
                const int64_t tq = (T.nq + bm - 1) / bm, nc = (T.nk + A.key_chunk - 1) / A.key_chunk;
                for (int64_t c = 0; c < nc; ++c) {
                    put_units(T, A, bm, c, units + at, tid & 63, 64);
                    at += tq - tile_min(T, A.p.causal, A.key_chunk, bm, c);
                }
            }
        __syncthreads();
    }
    if (tid == 0) *gp(count) = carry;
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uni64(int64_t x) {
    return (int64_t)(((uint64_t)(uint32_t)uni((int)(x >> 32)) << 32) | (uint32_t)uni((int)x));
}

// 16-byte pieces ("chunks") of a row: EPC elements each. A pair of chunks, one
// for each half of the wave, feeds one bf16 or four float32 matrix
// instructions: lane l of a 32 x 32 operand holds row l % 32 and half l / 32 of
// the instruction's k, and which k an instruction multiplies is free as long as
// both operands agree.
template <typename T> struct Frag;
template <> struct Frag<bf16> {
    typedef bf16x8 V;
    static constexpr int EPC = 8;
    static __device__ __forceinline__ f32x16 mma(V a, V b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Frag<float> {
    typedef f32x4 V;
    static constexpr int EPC = 4;
    static __device__ __forceinline__ f32x16 mma(V a, V b, f32x16 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

// How rows lie: RAGGED element by element at any alignment and dim; PADDED and
// FULL in whole 16-byte chunks, fewer than (exactly) the instance's width.
enum : int { RAGGED = 0, PADDED = 1, FULL = 2 };

// Chunk c of a row of dim elements, zeros from element dim on.
template <typename T, int ROWS>
__device__ __forceinline__ typename Frag<T>::V load_chunk(const MU_GLOBAL T* row, int c, int dim) {
    typename Frag<T>::V v;
    constexpr int EPC = Frag<T>::EPC;
    if constexpr (ROWS == FULL) return *(const MU_GLOBAL typename Frag<T>::V*)(row + c * EPC);
#pragma unroll
    for (int e = 0; e < EPC; ++e) v[e] = (T)0.f;
    if constexpr (ROWS == PADDED) {
        if (c * EPC < dim) v = *(const MU_GLOBAL typename Frag<T>::V*)(row + c * EPC);
    } else {
#pragma unroll
        for (int e = 0; e < EPC; ++e)
            if (c * EPC + e < dim) v[e] = row[c * EPC + e];
    }
    return v;
}

// max(|a|, |b|, m) that keeps NaN
__device__ __forceinline__ float absmax3(float a, float b, float m) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b)), m);
}

// Logits of a query tile against a stream of key tiles. Four waves of MT * 32
// queries each keep their queries in registers (the left operand of every
// product); the keys pass through a ring of NS LDS slots of BN rows, read as
// right operands by all four. Nothing but a running maximum leaves the matrix
// instructions, one max3 for two logits.
//
// A slot holds BN rows of NC chunks; chunk c of row r lies at position
// c ^ ((r >> SH) & (GR - 1)) of its row, which spreads the 16 lanes that read
// one chunk column of 16 rows over all 16 positions of 256 bytes: no bank
// conflicts at any NC. FULL and PADDED rows go from memory straight into the
// slot (the lane's address carries the permutation; chunks beyond dim are zeroed
// once and never written), RAGGED ones pass through registers.
//
// Rows past the end of a sequence read its last row again, which cannot change
// a maximum; only tiles that the causal border crosses test each pair.
template <typename T, int DP, int BN, int MT, int NS, int ROWS>
__global__ __launch_bounds__(NTHR, 2) void k_qkmax(QkMaxArgs A) {
    typedef typename Frag<T>::V V;
    constexpr bool DIRECT = ROWS != RAGGED;
    constexpr int EPC = Frag<T>::EPC, NC = DP / EPC, NK = NC / 2, ROWB = NC * 16, BM = 4 * MT * 32;
    constexpr int GR = NC % 16 == 0 ? 16 : NC % 8 == 0 ? 8 : NC % 4 == 0 ? 4 : 2;
    constexpr int SH = GR == 16 ? 0 : GR == 8 ? 1 : GR == 4 ? 2 : 3;
    constexpr int SLOTS = BN * NC;                     // chunks of a tile
    constexpr int NL = (SLOTS / 64 + 3) / 4;           // direct loads of a wave and tile
    static_assert(SLOTS % 64 == 0, "whole loads");
    constexpr int TB = BN * ROWB;
    __shared__ __align__(256) char s0[TB], s1[TB], s2[TB];
    static_assert(NS == 3, "three slots");
    __shared__ int red[4];
    const mu_qk_logits& P = A.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), l32 = lane & 31, half = lane >> 5;
    const int G = P.q_heads / P.k_heads;

    // chunk positions of this lane's reads: RA of them, then a multiple of GR * 16 bytes further
    constexpr int RA = GR / 2 < NK ? GR / 2 : NK;
    int rd[RA];
    const int sw = (l32 >> SH) & (GR - 1);
#pragma unroll
    for (int k = 0; k < RA; ++k) rd[k] = l32 * ROWB + (((2 * k + half) ^ sw) * 16);
    // this lane's part of each load: row and chunk
    int lrow[NL], lchk[NL], lpos[NL];
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        lpos[j] = uni(min(wave + 4 * j, SLOTS / 64 - 1));   // a last odd load is done twice
        const int q = lpos[j] * 64 + lane;
        lrow[j] = q / NC;
        lchk[j] = (q % NC) ^ ((lrow[j] >> SH) & (GR - 1));
    }
    if constexpr (ROWS == PADDED) {
        for (int i = tid; i < TB / 16; i += NTHR) {
            ((LDSP f32x4*)(LDSP char*)s0)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            ((LDSP f32x4*)(LDSP char*)s1)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            ((LDSP f32x4*)(LDSP char*)s2)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        __syncthreads();
    }

    const int64_t per_head = *gp(A.count), total = per_head * P.q_heads;
    // XCD x works on units [x * total / 8, (x + 1) * total / 8) of the order
    // key head, record, query head: what runs together there shares its keys
    const int xcd = blockIdx.x & 7, stride = gridDim.x >> 3;
    const int64_t u_end = total * (xcd + 1) / 8;
    int64_t u = total * xcd / 8 + (blockIdx.x >> 3);
    auto record = [&](int64_t x) { return (x < u_end ? x : u_end - 1) % (per_head * G) / G; };
    if (u >= u_end) return;
    Unit nxt = A.units[record(u)];
    for (; u < u_end; u += stride) {
        const int64_t q_off = uni64(nxt.q_off), k_off = uni64(nxt.k_off);
        const int nrows = uni(nxt.rows), nkeys = uni(nxt.keys), see = uni(nxt.see);
        nxt = A.units[record(u + stride)];   // needed a unit later
        const int hk = (int)(u / (per_head * G)), h = hk * G + (int)(u % G);
        const MU_GLOBAL T* kbase = (const MU_GLOBAL T*)P.k + k_off + hk * P.k_stride_h;
        const int ntiles = (nkeys + BN - 1) / BN;

        auto stage = [&](char* slot, int kt) {
            const int rem = nkeys - kt * BN;   // rows left from this tile on
            const MU_GLOBAL T* base = kbase + (int64_t)kt * BN * P.k_stride_s;
            if constexpr (DIRECT) {
                const int sb = (int)P.k_stride_s * (int)sizeof(T);
                const __amdgpu_buffer_rsrc_t rs =
                    __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (BN - 1) * sb + P.dim * (int)sizeof(T), BUF_RAW32);
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    const int vo = min(lrow[j], rem - 1) * sb + lchk[j] * 16;
                    if (ROWS == FULL || lchk[j] * EPC < P.dim)
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDSP void*)(slot + lpos[j] * 1024), 16, vo, 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    const MU_GLOBAL T* row = base + (int64_t)min(lrow[j], rem - 1) * P.k_stride_s;
                    *(LDSP V*)((LDSP char*)slot + lpos[j] * 1024 + lane * 16) = load_chunk<T, RAGGED>(row, lchk[j], P.dim);
                }
            }
        };

        // this wave's queries; how many of the keys its last and its first row see
        const int w_row = wave * (MT * 32);
        const bool live = w_row < nrows;
        const int see_last = !live ? 0 : min(nkeys, see + min(w_row + MT * 32, nrows) - 1);
        const int see_all = see + w_row;
        stage(s0, 0);
        if (ntiles > 1) stage(s1, 1);
        V qf[MT][NK];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int i = min(w_row + m * 32 + l32, nrows - 1);
            const MU_GLOBAL T* row = (const MU_GLOBAL T*)P.q + q_off + (int64_t)i * P.q_stride_s + h * P.q_stride_h;
#pragma unroll
            for (int k = 0; k < NK; ++k) qf[m][k] = load_chunk<T, ROWS>(row, 2 * k + half, P.dim);
        }

        float best = 0.f;
        auto compute = [&](const char* slot, int kt) {
            if (kt * BN >= see_last) return;
            const bool border = min((kt + 1) * BN, nkeys) > see_all;
#pragma unroll
            for (int n = 0; n < BN / 32; ++n) {
                f32x16 acc[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[m][e] = 0.f;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    const V kf = *(const LDSP V*)((const LDSP char*)slot + rd[k % RA] + n * 32 * ROWB + k / RA * (RA * 32));
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[m] = Frag<T>::mma(qf[m][k], kf, acc[m]);
                }
                if (border) {
                    const int j = min(kt * BN + n * 32 + l32, nkeys - 1) - see;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int i = min(w_row + m * 32 + 8 * (e / 4) + 4 * half + e % 4, nrows - 1);
                            acc[m][e] = j < i ? acc[m][e] : 0.f;
                        }
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) best = absmax3(acc[m][e], acc[m][e + 1], best);
            }
        };
        // Tile kt in slot kt % 3. The wait leaves the loads of the tile behind
        // it in flight (counted where every wave issues the same number); past
        // the barrier every wave has finished tile kt - 1, whose slot the next
        // loads take.
        auto step = [&](char* cur, char* nxt_slot, int kt) {
            if (ROWS == FULL && kt + 1 < ntiles) MU_WAIT_VMCNT_LGKM0(NL);
            else MU_WAIT_VMCNT_LGKM0(0);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (kt + 2 < ntiles) stage(nxt_slot, kt + 2);
            compute(cur, kt);
        };
        for (int kt = 0; kt < ntiles; kt += 3) {
            step(s0, s2, kt);
            if (kt + 1 < ntiles) step(s1, s0, kt + 1);
            if (kt + 2 < ntiles) step(s2, s1, kt + 2);
        }
        int bits = __float_as_int(best) & 0x7fffffff;
        for (int o = 32; o >= 1; o >>= 1) bits = max(bits, __shfl_xor(bits, o, 64));
        if (lane == 0) red[wave] = bits;
        __syncthreads();   // also: every wave is done with the slots
        if (tid == 0) {
            bits = max(max(red[0], red[1]), max(red[2], red[3]));
            if (bits) atomicMax((int*)P.max_logit + h, __float_as_int(__builtin_fabsf(P.scale) * __int_as_float(bits)) & 0x7fffffff);
        }
    }
}

template <typename T, int DP, int BN, int MT, int NS>
hipError_t launch(const QkMaxArgs& a, bool direct, int grid, hipStream_t s) {
    if (!direct) hipLaunchKernelGGL((k_qkmax<T, DP, BN, MT, NS, RAGGED>), dim3(grid), dim3(NTHR), 0, s, a);
    else if (a.p.dim < DP) hipLaunchKernelGGL((k_qkmax<T, DP, BN, MT, NS, PADDED>), dim3(grid), dim3(NTHR), 0, s, a);
    else hipLaunchKernelGGL((k_qkmax<T, DP, BN, MT, NS, FULL>), dim3(grid), dim3(NTHR), 0, s, a);
    return hipGetLastError();
}

// Instances by padded head width.
struct Shape {
    int dp, bn, bm;
};
Shape shape_of(int dtype, int dim) {
    const int dp = dim <= 32 ? 32 : dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256;
    if (dtype == MU_BF16) return {dp, dp <= 128 ? 64 : 32, 256};
    return {dp, 32, dp <= 128 ? 256 : 128};
}
hipError_t launch_shape(const QkMaxArgs& a, int dp, bool direct, int grid, hipStream_t s) {
    if (a.p.dtype == MU_BF16) switch (dp) {
        case 32: return launch<bf16, 32, 64, 2, 3>(a, direct, grid, s);
        case 64: return launch<bf16, 64, 64, 2, 3>(a, direct, grid, s);
        case 96: return launch<bf16, 96, 64, 2, 3>(a, direct, grid, s);
        case 128: return launch<bf16, 128, 64, 2, 3>(a, direct, grid, s);
        case 192: return launch<bf16, 192, 32, 2, 3>(a, direct, grid, s);
        default: return launch<bf16, 256, 32, 2, 3>(a, direct, grid, s);
    }
    switch (dp) {
        case 32: return launch<float, 32, 32, 2, 3>(a, direct, grid, s);
        case 64: return launch<float, 64, 32, 2, 3>(a, direct, grid, s);
        case 96: return launch<float, 96, 32, 2, 3>(a, direct, grid, s);
        case 128: return launch<float, 128, 32, 2, 3>(a, direct, grid, s);
        case 192: return launch<float, 192, 32, 1, 3>(a, direct, grid, s);
        default: return launch<float, 256, 32, 1, 3>(a, direct, grid, s);
    }
}

int check(const mu_qk_logits* a) {
    if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
    if (a->dtype != MU_F32 && a->dtype != MU_BF16) return fail(MU_ERR_DTYPE, "unknown dtype %d", a->dtype);
    if (a->batch < 0 || a->batch > (1 << 24) || a->q_len < 0 || a->k_len < 0 || a->q_len > 0x7fffff00LL || a->k_len > 0x7fffff00LL)
        return fail(MU_ERR_INVALID_ARG, "bad batch or length");
    if (a->q_heads < 1 || a->q_heads > (1 << 20) || a->k_heads < 1 || a->q_heads % a->k_heads != 0)
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

// What a call launches.
struct Plan {
    Shape sh;
    int64_t key_chunk;
    int64_t most;      // units of one head at most
    size_t bytes;      // of workspace
};
Plan plan_of(const mu_qk_logits* a) {
    Plan p;
    p.sh = shape_of(a->dtype, a->dim);
    const int64_t seqs = std::max<int64_t>(1, a->batch), bm = p.sh.bm;
    const int64_t tiles = a->cu_q ? a->q_len / bm + seqs : seqs * ((a->q_len + bm - 1) / bm);
    const int64_t keys = a->cu_q ? (a->k_len + seqs - 1) / seqs : a->k_len;   // of a sequence, about
    // Key chunk: a few units for each workgroup slot, between 256 and 4096 keys.
    p.key_chunk = 4096;
    while (p.key_chunk > 256 && tiles * a->q_heads * ((keys + p.key_chunk - 1) / p.key_chunk) < 8 * 2 * 256) p.key_chunk /= 2;
    p.most = tiles * ((a->k_len + p.key_chunk - 1) / p.key_chunk);
    p.bytes = ALIGN + align_up(sizeof(Unit) * (size_t)p.most);
    return p;
}

}  // namespace

extern "C" {

int mu_qk_max_logits_workspace_size(const mu_qk_logits* a, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check(a);
        if (rc) return rc;
        *bytes = plan_of(a).bytes;
        return MU_OK;
    });
}

int mu_qk_max_logits(const mu_qk_logits* a, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check(a);
        if (rc) return rc;
        const bool empty = a->batch == 0 || a->q_len == 0 || a->k_len == 0;
        if (empty && a->accumulate) return MU_OK;
        const Plan pl = plan_of(a);
        const Shape sh = pl.sh;
        if (!ws) return fail(MU_ERR_WORKSPACE, "workspace is null (need %zu bytes)", pl.bytes);
        if (!aligned(ws, ALIGN)) return fail(MU_ERR_WORKSPACE, "workspace must be 256-byte aligned");
        if (ws_bytes < pl.bytes) return fail(MU_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, pl.bytes);
        hipStream_t s = (hipStream_t)stream;
        const int es = a->dtype == MU_BF16 ? 2 : 4;
        // rows as whole 16-byte chunks, a tile of them within 32-bit offsets
        const int64_t mix = a->q_stride_b | a->q_stride_s | a->q_stride_h | a->k_stride_b | a->k_stride_s | a->k_stride_h | a->dim;
        const bool direct = (mix * es) % 16 == 0 && aligned(a->q, 16) && aligned(a->k, 16) &&
                            a->k_stride_s < ((int64_t)1 << 30) / (sh.bn * es);
        int64_t* count = (int64_t*)ws;
        Unit* units = (Unit*)((char*)ws + ALIGN);
        const QkMaxArgs q{*a, count, units, pl.key_chunk};
        rc = timed_launch(MU_K_QKMAX, 0.0, 0.0, s, [&] {
            hipLaunchKernelGGL(k_qk_plan, dim3(1), dim3(PLAN_THR), 0, s, q, count, units, sh.bm);
            return hipGetLastError();
        }, "max logits plan");
        if (rc || empty) return rc;
        int cus = 0;
        rc = cu_count(&cus);
        if (rc) return rc;
        const double nb = a->cu_q ? 1 : a->batch;
        const double bytes = nb * a->dim * es * ((double)a->q_len * a->q_heads + (double)a->k_len * a->k_heads);
        const double flops = 2.0 * nb * (double)a->q_len * (double)a->k_len * a->q_heads * a->dim * (a->causal ? 0.5 : 1.0);
        const int grid = (int)std::min<int64_t>(2 * (int64_t)cus, (pl.most * a->q_heads + 7) / 8 * 8);
        return timed_launch(MU_K_QKMAX, flops, bytes, s, [&] { return launch_shape(q, sh.dp, direct, grid, s); },
                            "max logits launch");
    });
}

}  // extern "C"
