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
#include <type_traits>
#include <vector>

#include "../../include/muon_mi355x.h"
#include "capi_common.hpp"
#include "common.hpp"

using namespace mu;

namespace {

constexpr int NTHR = 256;

#define LDSP __attribute__((address_space(3)))
// s_waitcnt with vmcnt(n); with vmcnt(n) and lgkmcnt(0) (gfx9 encoding)
#define MU_WAIT_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (15 << 8) | (((n) >> 4) << 14))
#define MU_WAIT_VMCNT_LGKM0(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (0 << 8) | (((n) >> 4) << 14))
constexpr int BUF_RAW32 = 0x00020000;   // word 3 of a raw buffer resource

typedef float f32x16 __attribute__((ext_vector_type(16)));

// The work is key tiles: query tile t (BM rows) of a sequence and head passes
// over the tiles of BN keys that its last row sees. All of them are laid out on
// one line (head slowest, then sequence, query tile, key tile), each query tile
// with COST more places in front for what it costs to begin and to end at the
// border, and every workgroup takes an equal run of the line, wherever that
// starts and ends. COST in tiles of bfloat16 and of float32, which take about
// three times as long: 6 and 2, the best of 1, 2, 3, 6 and 12 (8192 tokens,
// 16 heads of 64: 66, 62, 62, 59, 61 us; 4 x 1024 tokens, 12 heads of 64 in
// float32: 37.4, 37.2, 38.4, 42.4, 51.4 us) and of 4, 6, 8, 10 and 14 (23 packed
// sequences: 68.8, 65.9, 69.1, 70.0, 75.7 us). The bfloat16 instances with tiles of
// 32 keys have the same 6, which is within 5 % of the best of 2, 3, 4, 6, 12 and 20
// (16 heads; one sequence of 8192 tokens: dim 100 290, 288, 289, 295, 308, 316 us,
// dim 192 173, 166, 163, 160, 159, 164, dim 256 243, 241, 237, 231, 223, 227; the 23
// packed sequences: 174, 168, 166, 168, 178, 205, then 91, 88, 85, 84, 85, 92 and
// 130, 126, 122, 120, 120, 128; 4 x 1024 tokens: 41, 41, 41, 43, 48, 53, then 25, 24,
// 22, 24, 24, 26 and 32, 31, 31, 31, 32, 33).
template <typename T> constexpr int COST_OF = sizeof(T) == 2 ? 6 : 2;
// How a workgroup finds its run: it takes all of a head; by arithmetic, as
// sequences are of one length; from up to 64 sequences, one a lane; from the
// places before each sequence that a launch before wrote.
enum : int { BY_HEAD = 0, ALIKE = 1, IN_LANES = 2, PREFIX = 3 };
struct QkMaxArgs {
    mu_qk_logits p;
    const int64_t* prefix;   // PREFIX: [batch + 1] places of one head before each sequence
    int plan;
};

struct Seq {
    int64_t q0, k0;   // element offset of its first row (without the head)
    int32_t nq, nk;
};

__device__ inline int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

__device__ inline Seq seq_of(const mu_qk_logits& A, int64_t b) {
    Seq s;
    if (A.cu_q) {
        const MU_GLOBAL int32_t* cq = (const MU_GLOBAL int32_t*)A.cu_q;
        const MU_GLOBAL int32_t* ck = A.cu_k ? (const MU_GLOBAL int32_t*)A.cu_k : cq;
        const int64_t a = clamp64(cq[b], 0, A.q_len), c = clamp64(ck[b], 0, A.k_len);
        s.nq = (int32_t)(clamp64(cq[b + 1], a, A.q_len) - a);
        s.nk = (int32_t)(clamp64(ck[b + 1], c, A.k_len) - c);
        s.q0 = a * A.q_stride_s;
        s.k0 = c * A.k_stride_s;
    } else {
        s.nq = (int32_t)(A.q_lengths ? clamp64(((const MU_GLOBAL int32_t*)A.q_lengths)[b], 0, A.q_len) : A.q_len);
        s.nk = (int32_t)(A.k_lengths ? clamp64(((const MU_GLOBAL int32_t*)A.k_lengths)[b], 0, A.k_len) : A.k_len);
        s.q0 = b * A.q_stride_b;
        s.k0 = b * A.k_stride_b;
    }
    return s;
}

// Key tiles of a sequence and head. Query tile t < last sees (t + 1) BM + nk - nq
// keys (causal), so (t + 1) BM / BN + o tiles with o = ceil((nk - nq) / BN) from
// the first t that sees any; the last one sees all keys.
template <int BM, int BN, int COST>
struct Tiles {
    int t0, last, all;   // first and last query tile with keys, tiles of all keys
    int o;
    bool causal;
    __device__ Tiles(const Seq& S, bool c) : causal(c) {
        // (lengths are below 2^31 - 256)
        last = (S.nq + BM - 1) / BM - 1;
        all = (S.nk + BN - 1) / BN;
        const int off = S.nk - S.nq;
        o = off >= 0 ? (off + BN - 1) / BN : -(-off / BN);
        t0 = causal && off < 0 ? (BM - off) / BM - 1 : 0;   // ceil((1 - off) / BM) - 1
        if (S.nq <= 0 || S.nk <= 0) t0 = 0, last = -1;
    }
    __device__ int of(int t) const { return causal && t < last ? (t + 1) * (BM / BN) + o : all; }
    // places of the query tiles before t, t0 <= t <= last
    __device__ int64_t before(int t) const {
        const int64_t n = t - t0, both = (int64_t)t + t0 + 1;   // t (t + 1) - t0 (t0 + 1) = n both
        return n * COST + (causal ? n * o + (BM / BN) * (n * both / 2) : n * all);
    }
    __device__ int64_t total() const { return last < 0 ? 0 : before(last) + COST + all; }
};

// One workgroup: zeros to take maxima from, and (PREFIX) the places before each
// sequence.
constexpr int PLAN_THR = 1024;
template <int BM, int BN, int COST>
__global__ __launch_bounds__(PLAN_THR) void k_qk_plan(QkMaxArgs A, int64_t* prefix) {
    __shared__ int64_t wsum[PLAN_THR / 64];
    const int tid = threadIdx.x;
    if (!A.p.accumulate)
        for (int i = tid; i < A.p.q_heads; i += PLAN_THR) gp(A.p.max_logit)[i] = 0.f;
    if (A.plan != PREFIX) return;
    int64_t carry = 0;
    for (int64_t b0 = 0; b0 < A.p.batch; b0 += PLAN_THR) {
        const int64_t b = b0 + tid;
        int64_t n = b < A.p.batch ? Tiles<BM, BN, COST>(seq_of(A.p, b), A.p.causal != 0).total() : 0;
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t up = __shfl_up(n, off, 64);
            if ((tid & 63) >= off) n += up;
        }
        if ((tid & 63) == 63) wsum[tid >> 6] = n;
        __syncthreads();
        int64_t before = carry;
        for (int w = 0; w < PLAN_THR / 64; ++w) {
            if (w < (tid >> 6)) before += wsum[w];
            carry += wsum[w];
        }
        if (b < A.p.batch) gp(prefix)[b + 1] = before + n;
        __syncthreads();
    }
    if (tid == 0) gp(prefix)[0] = 0;
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

// How rows lie: RAGGED at any alignment and dim; PADDED and
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
        // gfx950 takes global vector accesses at any address
        typedef typename Frag<T>::V VU __attribute__((aligned(sizeof(T))));
        if ((c + 1) * EPC <= dim) v = *(const MU_GLOBAL VU*)(row + c * EPC);
        else if (c * EPC < dim) {
#pragma unroll
            for (int e = 0; e < EPC; ++e)
                if (c * EPC + e < dim) v[e] = row[c * EPC + e];
        }
    }
    return v;
}

// max(|a|, |b|, m) that keeps NaN
__device__ __forceinline__ float absmax3(float a, float b, float m) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b)), m);
}

// Logits of a query tile against a stream of key tiles. Four waves of MT * 32
// queries each keep their queries in registers (the left operand of every
// product); the keys pass through a ring of four LDS slots of BN rows, read as
// right operands by all four. Nothing but a running maximum leaves the matrix
// instructions, one max3 for two logits.
//
// A slot holds BN rows of NC chunks; chunk c of row r lies at position
// c ^ ((r >> SH) & (GR - 1)) of its row, which spreads the 16 lanes that read
// one chunk column of 16 rows over all 16 positions of 256 bytes: no bank
// conflicts at any NC. FULL and PADDED rows go from memory straight into the
// slot (the lane's address carries the permutation; chunks beyond dim are zeroed
// once, and their loads lie outside the buffer resource, which gives zeros),
// RAGGED ones pass through registers.
//
// Rows past the end of a sequence read its last row again, which cannot change
// a maximum; only tiles that the causal border crosses test each pair.
//
// Bound by the matrix instructions: 8192 tokens, 32 heads of 128 on 8 key heads,
// causal, take 203-219 us, 1.26-1.35 PFLOP/s of the visible pairs (a library
// product of 8192^3 reaches 1.19 on the same card; the clock falls under this
// load). float32 reaches 127 TFLOP/s at 4096 tokens, 12 heads of 64 (library
// product 153). Short sequences are bound by what a query tile costs to begin:
// 23 packed sequences of 16384 tokens, 16 heads of 128, 64 us, 0.72 PFLOP/s.
template <typename T, int DP, int BN, int MT, int WPE, int ROWS>
__global__ __launch_bounds__(NTHR, WPE) void k_qkmax(QkMaxArgs A) {
    typedef typename Frag<T>::V V;
    constexpr bool DIRECT = ROWS != RAGGED;
    constexpr int COST = COST_OF<T>, EPC = Frag<T>::EPC, NC = DP / EPC, NK = NC / 2, ROWB = NC * 16, BM = 4 * MT * 32;
    constexpr int GR = NC % 16 == 0 ? 16 : NC % 8 == 0 ? 8 : NC % 4 == 0 ? 4 : 2;
    constexpr int SH = GR == 16 ? 0 : GR == 8 ? 1 : GR == 4 ? 2 : 3;
    constexpr int SLOTS = BN * NC;                     // chunks of a tile
    constexpr int NL = SLOTS / 256;                    // direct loads of a wave and tile
    static_assert(SLOTS % 256 == 0, "the same number of whole loads for each wave");
    constexpr int TB = BN * ROWB, NB = BN / 32;
    constexpr int PD = NK <= 8 ? NK : NK % 8 == 0 ? 8 : 6;
    static_assert(NK % PD == 0, "a column block is whole rounds of the operand ring");
    __shared__ __align__(256) char s0[TB], s1[TB], s2[TB], s3[TB];
    __shared__ int red[4];
    const mu_qk_logits& P = A.p;
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, half = lane >> 5;
    int wave = uni(tid >> 6);
    // its range is hidden: where the compiler can tell a read of the upper rows
    // of a slot from the slot's first direct load, it no longer connects it to
    // the slot's others and waits for every load in flight
    asm("" : "+s"(wave));
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
        lpos[j] = wave + 4 * j;
        const int q = lpos[j] * 64 + lane;
        lrow[j] = q / NC;
        lchk[j] = (q % NC) ^ ((lrow[j] >> SH) & (GR - 1));
    }
    if constexpr (ROWS == PADDED) {
        for (int i = tid; i < TB / 16; i += NTHR) {
            ((LDSP f32x4*)(LDSP char*)s0)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            ((LDSP f32x4*)(LDSP char*)s1)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            ((LDSP f32x4*)(LDSP char*)s2)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            ((LDSP f32x4*)(LDSP char*)s3)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        __syncthreads();
    }

    const int PLAN = A.plan;
    const bool by_head = PLAN == BY_HEAD;
    int64_t u = 0, u_end = (int64_t)1 << 60, r = 0, b = 0;
    int h = blockIdx.x, t = 0;
    if (!by_head) {
        // places before each sequence (the first 64 candidates of the search
        // below): of one length, of up to 64 in a wave's lanes, or from memory
        int64_t st = (P.batch + 63) / 64, cand = 0, each = 0, per_head;
        if (PLAN == ALIKE) {
            each = Tiles<BM, BN, COST>(seq_of(P, 0), P.causal != 0).total();
            per_head = each * P.batch;
        } else if (PLAN == IN_LANES) {
            const int64_t own = lane < P.batch ? Tiles<BM, BN, COST>(seq_of(P, lane), P.causal != 0).total() : 0;
            cand = own;
            for (int o = 1; o < 64; o <<= 1) {
                const int64_t up = __shfl_up(cand, o, 64);
                if (lane >= o) cand += up;
            }
            per_head = uni64(__shfl(cand, 63, 64));
            cand -= own;
        } else {
            const int64_t at = min<int64_t>(st * lane, P.batch - 1);
            cand = gp(A.prefix)[at];
            per_head = uni64(gp(A.prefix)[P.batch]);
        }
        const int64_t total = per_head * P.q_heads;
        // XCD x takes places [x * total / 8, (x + 1) * total / 8), so few key heads
        const int xcd = blockIdx.x & 7, wgs = gridDim.x >> 3, w_in = blockIdx.x >> 3;
        const int64_t x_lo = total * xcd / 8, x_n = total * (xcd + 1) / 8 - x_lo;
        u = x_lo + x_n * w_in / wgs;
        u_end = x_lo + x_n * (w_in + 1) / wgs;
        if (u >= u_end) return;
        h = (int)(u / per_head);
        r = u - h * per_head;   // place in the head
        // its sequence: the last one that starts at or before r, 64 candidates at a time
        int64_t before = 0;
        if (PLAN == ALIKE) {
            b = r / each;
            before = b * each;
        } else {
            for (int64_t n = P.batch; n > 1;) {
                const int k = __popcll(__ballot(lane * st < n && cand <= r));   // >= 1
                before = uni64(__shfl(cand, k - 1, 64));
                b += (k - 1) * st;
                n = min<int64_t>(st, n - (k - 1) * st);
                st = (n + 63) / 64;
                const int64_t next = b + min<int64_t>(st * lane, n - 1);
                if (n > 1) cand = gp(A.prefix)[next];
            }
            b = uni64(b);
        }
        r -= before;
    }
    const bool none = P.batch == 0 || P.q_len == 0 || P.k_len == 0;   // (lengths are not read then)
    Seq S{0, 0, 0, 0};
    if (!none) S = seq_of(P, b);
    Tiles<BM, BN, COST> tl(S, P.causal != 0);
    if (by_head && !none)
        while (tl.last < 0 && ++b < P.batch) {
            S = seq_of(P, b);
            tl = Tiles<BM, BN, COST>(S, P.causal != 0);
        }
    t = tl.t0;
    for (int n = tl.last - tl.t0 + 1; !by_head && n > 1;) {   // the query tile of place r
        const int half_n = n / 2;
        if (tl.before(t + half_n) <= r) t += half_n, n -= half_n;
        else n = half_n;
    }
    if (!by_head) r -= tl.before(t);
    bool more = tl.last >= 0;   // (false: by head, and no sequence has a tile)
    // the largest magnitude of head h, kept over its query tiles
    float best = 0.f;
    auto flush = [&] {
        int bits = __float_as_int(best) & 0x7fffffff;
        for (int o = 32; o >= 1; o >>= 1) bits = max(bits, __shfl_xor(bits, o, 64));
        if (lane == 0) red[wave] = bits;
        __syncthreads();
        if (tid == 0) {
            bits = max(max(red[0], red[1]), max(red[2], red[3]));
            bits = __float_as_int(__builtin_fabsf(P.scale) * __int_as_float(bits)) & 0x7fffffff;
            int* out = (int*)P.max_logit + h;
            if (!by_head) atomicMax(out, bits);
            else *gp(out) = P.accumulate ? max(*gp(out), bits) : bits;
        }
        __syncthreads();   // (a run that ends before its next head's first tile flushes twice in a row)
        best = 0.f;
    };
    for (; more; r = 0) {
        // key tiles first .. first + ntiles - 1 of query tile t, from its place r on
        const int64_t places = min<int64_t>(COST + tl.of(t) - r, u_end - u);
        u += places;
        const int first = (int)max<int64_t>(r - COST, 0), ntiles = (int)max<int64_t>(r + places - COST, 0) - first;
        if (ntiles <= 0) break;   // the run ends before the first tile
        const int hk = h / G;
        const int k_lo = first * BN, off = S.nk - S.nq;
        const int nrows = min(BM, S.nq - t * BM);
        const int k_hi = P.causal ? min(S.nk, t * BM + nrows + off) : S.nk;
        const int nkeys = min(k_hi - k_lo, ntiles * BN);
        // row i sees the run's keys j < see + i; not causal, all of them
        const int see = P.causal ? min(max(t * BM + 1 + off - k_lo, -BM), nkeys) : nkeys;
        const int64_t q_off = S.q0 + (int64_t)t * BM * P.q_stride_s;
        const MU_GLOBAL T* kbase = (const MU_GLOBAL T*)P.k + S.k0 + hk * P.k_stride_h + (int64_t)k_lo * P.k_stride_s;

        // Tiles past the last one are the last one again: every wave then has
        // the same number of loads in flight at every wait.
        auto stage = [&](char* slot, int kt) {
            kt = min(kt, ntiles - 1);
            const int rem = nkeys - kt * BN;   // rows left from this tile on
            const MU_GLOBAL T* base = kbase + (int64_t)kt * BN * P.k_stride_s;
            if constexpr (DIRECT) {
                const int sb = (int)P.k_stride_s * (int)sizeof(T);
                const __amdgpu_buffer_rsrc_t rs =
                    __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (BN - 1) * sb + P.dim * (int)sizeof(T), BUF_RAW32);
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    int vo = min(lrow[j], rem - 1) * sb + lchk[j] * 16;
                    if (ROWS == PADDED && lchk[j] * EPC >= P.dim) vo = 0x7fffff00;   // beyond the resource: reads nothing
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

        // this wave's queries; how many of the keys its last row sees
        const int w_row = wave * (MT * 32);
        const bool live = w_row < nrows;
        const int see_last = !live ? 0 : min(nkeys, see + min(w_row + MT * 32, nrows) - 1);
        stage(s0, 0);
        stage(s1, 1);
        V qf[MT][NK];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int i = min(w_row + m * 32 + l32, nrows - 1);
            const MU_GLOBAL T* row = (const MU_GLOBAL T*)P.q + q_off + (int64_t)i * P.q_stride_s + h * P.q_stride_h;
#pragma unroll
            for (int k = 0; k < NK; ++k) qf[m][k] = load_chunk<T, ROWS>(row, 2 * k + half, P.dim);
        }

        // The stream of right operands: tile after tile, 32 keys (a column
        // block) after 32 keys, chunk pair after chunk pair. f holds the next
        // PD of them; each place is read again as soon as its matrix
        // instructions have issued, so a read has PD * MT of those to arrive.
        // Accumulators alternate between column blocks, and the maximum of one
        // block is taken while the next is multiplied.
        V f[PD];
        f32x16 acc[2][MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[0][m][e] = acc[1][m][e] = 0.f;
        auto operand = [&](const char* slot, int n, int k) {
            return *(const LDSP V*)((const LDSP char*)slot + rd[k % RA] + n * 32 * ROWB + k / RA * (RA * 32));
        };
        // The maximum over a block of logits. A lane's element e of block m is
        // row 32 m + 8 (e / 4) + e % 4 (from a base of its own) of one key; MASK:
        // only rows beyond `thr` see it.
        auto take = [&](auto mask, f32x16 (&c)[MT], int thr) {
            if constexpr (decltype(mask)::value) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 16; ++e) c[m][e] = thr < m * 32 + 8 * (e / 4) + e % 4 ? c[m][e] : 0.f;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 16; e += 2) best = absmax3(c[m][e], c[m][e + 1], best);
        };
        // Makes tile kt readable (slot kt % 4) and sends for tile kt + 2, whose
        // slot tile kt - 2 has left: a wave that comes here has multiplied what
        // it read of that tile. The wait leaves the loads of tile kt + 1, and a
        // direct instance's reads of tile kt - 1, in flight.
        auto advance = [&](char* slot2, int kt) {
            if constexpr (DIRECT) MU_WAIT_VMCNT(NL);
            else MU_WAIT_VMCNT_LGKM0(0);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            stage(slot2, kt + 2);
        };
        // One tile. MASK: the causal border may cross it. (Rows past nrows and
        // keys past nkeys repeat the last ones; the last row sees every key of
        // the run, so neither needs a test of its own.)
        constexpr int SEE_ALL = -(1 << 30);
        int thr_prev = SEE_ALL;
        const int thr_lane = l32 - see - w_row - 4 * half;
        auto tile = [&](auto mask, const char* cur, const char* nxt_slot, char* slot2, int kt) {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                f32x16 (&c)[MT] = acc[NB == 1 ? 0 : n & 1];
                f32x16 (&prev)[MT] = acc[NB == 1 ? 1 : (n & 1) ^ 1];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 16; ++e) c[m][e] = 0.f;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    if (n == NB - 1 && k == NK - PD) advance(slot2, kt + 1);
#pragma unroll
                    for (int m = 0; m < MT; ++m) c[m] = Frag<T>::mma(qf[m][k], f[k % PD], c[m]);
                    const bool far = k + PD >= NK;
                    f[k % PD] = operand(n == NB - 1 && far ? nxt_slot : cur, far ? (n + 1) % NB : n, (k + PD) % NK);
                }
                const int thr = kt * BN + n * 32 + thr_lane;
                if constexpr (NB > 1) {
                    take(mask, prev, thr_prev);
                    // the maxima spread behind matrix instructions, from the
                    // second round on (the first waits for prev's last ones)
#pragma unroll
                    for (int k = 0; k < NK && !decltype(mask)::value; ++k) {
                        __builtin_amdgcn_sched_group_barrier(0x008, MT * (sizeof(T) == 2 ? 1 : 4), 0);
                        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        if (k > 0) __builtin_amdgcn_sched_group_barrier(0x002, (8 * MT + NK - 2) / (NK - 1), 0);
                    }
                } else {
                    take(mask, c, thr);
                }
                if (decltype(mask)::value) thr_prev = thr;
            }
        };
        // Tiles that all of the workgroup's rows see whole go four at a time
        // without a branch in between, then the others. The code keeps to
        // straight runs: where paths meet the compiler forgets which slot a
        // load in flight goes to and waits for all of them before the next read
        // (at the heads of the two loops here). A wave whose rows see nothing
        // further leaves, and only takes its part in loads and barriers.
        advance(s2, 0);
#pragma unroll
        for (int k = 0; k < PD; ++k) f[k] = operand(s0, 0, k);
        const int nwhole = see >= nkeys ? ntiles : max(see, 0) / BN;
        int kt = 0;
        for (; kt + 4 <= nwhole; kt += 4) {
            tile(std::false_type{}, s0, s1, s3, kt);
            tile(std::false_type{}, s1, s2, s0, kt + 1);
            tile(std::false_type{}, s2, s3, s1, kt + 2);
            tile(std::false_type{}, s3, s0, s2, kt + 3);
        }
        for (;;) {
            if (kt * BN >= see_last) break;
            tile(std::true_type{}, s0, s1, s3, kt);
            if (++kt * BN >= see_last) break;
            tile(std::true_type{}, s1, s2, s0, kt);
            if (++kt * BN >= see_last) break;
            tile(std::true_type{}, s2, s3, s1, kt);
            if (++kt * BN >= see_last) break;
            tile(std::true_type{}, s3, s0, s2, kt);
            ++kt;
        }
        if constexpr (NB > 1) take(std::true_type{}, acc[1], thr_prev);
        for (; kt < ntiles; ++kt) advance(kt % 4 == 0 ? s3 : kt % 4 == 1 ? s0 : kt % 4 == 2 ? s1 : s2, kt + 1);
        __syncthreads();   // every wave is done with the slots
        // the next query tile, sequence or head
        more = u < u_end;
        if (!more || ++t <= tl.last) continue;
        do {
            if (++b == P.batch) {
                if (by_head) {
                    more = false;
                    break;
                }
                flush();
                b = 0, ++h;
            }
            S = seq_of(P, b);
            tl = Tiles<BM, BN, COST>(S, P.causal != 0);
        } while (tl.last < 0);   // (not by head: a later sequence has tiles, as u < u_end)
        t = tl.t0;
    }
    flush();
}

// Pairs of nq queries and nk keys that count: query i sees min(nk, i + 1 + nk - nq) keys.
double visible_pairs(double nq, double nk, bool causal) {
    if (!causal) return nq * nk;
    const double n = std::min(nq, nk);   // the last n queries see nk - n + 1 .. nk keys
    return n * (nk - n) + n * (n + 1) / 2;
}

// Places of a head at most (lengths on the device may leave fewer).
double most_places(const mu_qk_logits* a, int bm, int bn, int cost) {
    const double q = a->cu_q ? (double)(a->q_len / bm) + a->batch : (double)a->batch * ((a->q_len + bm - 1) / bm);
    return a->q_len == 0 || a->k_len == 0 ? 0.0 : q * (cost + (double)((a->k_len + bn - 1) / bn));
}

// Reading the lengths in every workgroup costs less than waiting for another
// launch to write them and then for two loads: 23 packed sequences 65.3 against
// 66.2 us; one sequence of 1024 tokens (float32, 12 heads of 64) 17.6 against 18.8.
int plan_of(const mu_qk_logits* a) {
    return !a->cu_q && !a->q_lengths && !a->k_lengths ? ALIKE : a->batch <= 64 ? IN_LANES : PREFIX;
}

// Where a head has no more places than this, a workgroup takes all of one: it
// needs no plan and stores its maximum itself, one launch instead of two. Whole
// calls, with and without (16 us is two launches from the host): 12 heads of
// 256 tokens (10 places) 13.5 and 16.1 us, 512 tokens in one workgroup (28
// places) 13.5, but 16.8 and 16.2 with 64 heads of 128, 4 x 128 (32 places)
// 18.6 and 16.2, in float32 4 x 64 (16 places) 17.0 and 16.2.
constexpr int by_head_places(int cost) { return 4 * cost; }

// Up to so many tiles for each of the workgroups that the chip holds (all keys
// counted for every query) one workgroup a compute unit is as fast or faster:
// there the chain of loads before the first tile is what a run waits for. Whole
// calls, with as many as the chip holds and with one: float32, 12 heads of 64,
// 1024 tokens (6 tiles) 17.6 and 16.3 us, 16 heads of 128 (8 tiles) 29.8 and
// 27.7; bfloat16, 16 heads of 128, 2048 tokens (8 tiles) 17.1 and 16.0; but 4 x
// 1024 tokens, 32 heads of 64 (16 tiles) 17.3 and 19.7, float32 12 heads (24
// tiles) 35.5 and 36.6.
constexpr int FEW_TILES = 12;
struct Call {
    const mu_qk_logits* p;
    int64_t* prefix;
    bool direct;
    double flops, bytes;
    hipStream_t s;
};

// An instance: padded head width, keys of a tile, queries of a wave in 32s, waves a SIMD.
template <typename T, int DP, int BN, int MT, int WPE, int ROWS>
int run(const Call& c) {
    constexpr int BM = 4 * MT * 32;
    const double places = most_places(c.p, BM, BN, COST_OF<T>);
    QkMaxArgs q{*c.p, c.prefix, BY_HEAD};
    int grid = c.p->q_heads;
    if (places > by_head_places(COST_OF<T>)) {
        q.plan = plan_of(c.p);
        int rc = MU_OK;
        if (q.plan == PREFIX || !c.p->accumulate)
            rc = timed_launch(MU_K_QKMAX, 0.0, 0.0, c.s, [&] {
                hipLaunchKernelGGL((k_qk_plan<BM, BN, COST_OF<T>>), dim3(1), dim3(PLAN_THR), 0, c.s, q, c.prefix);
                return hipGetLastError();
            }, "max logits plan");
        if (rc) return rc;
        int cus = 0;
        rc = cu_count(&cus);
        if (rc) return rc;
        // as many workgroups as the chip holds at a time, one a compute unit
        // where that leaves them few tiles, fewer where there cannot be as many
        // tiles; the same number on each of the 8 XCDs
        const double tiles = most_places(c.p, BM, BN, 0) * c.p->q_heads;
        const int wgs = std::max(cus * (tiles <= (double)FEW_TILES * WPE * cus ? 1 : WPE) / 8, 1) * 8;
        grid = (int)std::min<double>(wgs, 8.0 * std::ceil(tiles / 8.0));
    }
    return timed_launch(MU_K_QKMAX, c.flops, c.bytes, c.s, [&] {
        hipLaunchKernelGGL((k_qkmax<T, DP, BN, MT, WPE, ROWS>), dim3(grid), dim3(NTHR), 0, c.s, q);
        return hipGetLastError();
    }, "max logits launch");
}

template <typename T, int DP, int BN, int MT, int WPE>
int run_direct(const Call& c) {
    return c.p->dim < DP ? run<T, DP, BN, MT, WPE, PADDED>(c) : run<T, DP, BN, MT, WPE, FULL>(c);
}

// The instances. bfloat16: 64 rows a wave, as a key read from LDS then feeds two
// matrix instructions (32 rows a wave 247 against 220 us at 8192 tokens, 32 heads
// of 128; 128 rows and one wave a SIMD 263), 64 keys a tile while four slots of
// them leave two workgroups a compute unit. float32 matrix instructions are so
// long that one operand read for each suffices: 32 rows a wave and 32 keys, whose
// finer tiles follow the causal border closer (12 heads of 64, 1024 tokens 18.6
// against 22.5 us). RAGGED rows pass through registers, so 32 keys a tile; 64
// rows a wave, as each piece that is loaded and stored then feeds two matrix
// instructions: dim 100, 16 heads, against 32 rows a wave, 4 x 2048 tokens 105 and
// 156 us, 8192 tokens 296 and 501, 1024 tokens 22.4 and 24.2, but 2 x 1024 tokens 31.6
// and 29.4. What bounds them: a tile's loads are stored to LDS at once, so every tile
// waits for memory, where direct loads stay in flight over two tiles. Their whole
// chunks are loaded as vectors at any address (dim 100, 2 x 1024 tokens, 32 rows a
// wave 27 us, 56 by elements).
int run_any(const Call& c) {
    const int d = c.p->dim;
    if (c.p->dtype == MU_BF16) {
        if (!c.direct)
            return d <= 64 ? run<bf16, 64, 32, 2, 2, RAGGED>(c) : d <= 128 ? run<bf16, 128, 32, 2, 2, RAGGED>(c)
                                                                          : run<bf16, 256, 32, 2, 1, RAGGED>(c);
        if (d <= 32) return run_direct<bf16, 32, 64, 2, 2>(c);
        if (d <= 64) return run_direct<bf16, 64, 64, 2, 2>(c);
        if (d <= 96) return run_direct<bf16, 96, 64, 2, 2>(c);
        if (d <= 128) return run_direct<bf16, 128, 64, 2, 2>(c);
        if (d <= 192) return run_direct<bf16, 192, 32, 2, 2>(c);
        return run_direct<bf16, 256, 32, 2, 1>(c);
    }
    if (!c.direct)
        return d <= 64 ? run<float, 64, 32, 1, 2, RAGGED>(c) : d <= 128 ? run<float, 128, 32, 1, 2, RAGGED>(c)
                                                                       : run<float, 256, 32, 1, 1, RAGGED>(c);
    if (d <= 32) return run_direct<float, 32, 32, 1, 2>(c);
    if (d <= 64) return run_direct<float, 64, 32, 1, 2>(c);
    if (d <= 96) return run_direct<float, 96, 32, 1, 2>(c);
    if (d <= 128) return run_direct<float, 128, 32, 1, 2>(c);
    if (d <= 192) return run_direct<float, 192, 32, 1, 1>(c);
    return run_direct<float, 256, 32, 1, 1>(c);
}

// The bytes that rows of (batch, len, heads, dim) elements at these strides span;
// false if they pass any memory.
bool span_of(const void* p, int64_t batch, int64_t sb, int64_t len, int64_t ss, int64_t heads, int64_t sh, int64_t dim,
             size_t es, std::vector<Range>& out) {
    if (batch <= 0 || len <= 0) return true;
    const double n = (double)(batch - 1) * (double)sb + (double)(len - 1) * (double)ss + (double)(heads - 1) * (double)sh + (double)dim;
    if (n > (double)((int64_t)1 << 50)) return false;
    const int64_t last = (batch - 1) * sb + (len - 1) * ss + (heads - 1) * sh + dim;
    out.push_back({(uintptr_t)p, (uintptr_t)p + (size_t)last * es, 0});
    return true;
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
    // max_logit is written first, so it may lie in no input
    std::vector<Range> in;
    const int64_t nb = a->cu_q ? 1 : a->batch;
    if (!span_of(a->q, nb, a->q_stride_b, a->q_len, a->q_stride_s, a->q_heads, a->q_stride_h, a->dim, es, in) ||
        !span_of(a->k, nb, a->k_stride_b, a->k_len, a->k_stride_s, a->k_heads, a->k_stride_h, a->dim, es, in))
        return fail(MU_ERR_INVALID_ARG, "strides are too large");
    for (const int32_t* p : {a->q_lengths, a->k_lengths, a->cu_q, a->cu_k})
        if (p) in.push_back({(uintptr_t)p, (uintptr_t)(p + a->batch + (a->cu_q ? 1 : 0)), 0});
    for (const Range& r : in)
        if (r.lo < (uintptr_t)(a->max_logit + a->q_heads) && (uintptr_t)a->max_logit < r.hi)
            return fail(MU_ERR_LAYOUT, "max_logit overlaps an input");
    return MU_OK;
}

// (the smallest tiles of the type's instances: a call that needs none by these
// counts needs none by its own)
size_t qk_workspace(const mu_qk_logits* a) {
    const int cost = a->dtype == MU_BF16 ? COST_OF<bf16> : COST_OF<float>;
    const bool few = most_places(a, 128, 32, cost) <= by_head_places(cost);
    return few || plan_of(a) != PREFIX ? 0 : align_up(sizeof(int64_t) * ((size_t)a->batch + 1));
}

}  // namespace

extern "C" {

int mu_qk_max_logits_workspace_size(const mu_qk_logits* a, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check(a);
        if (rc) return rc;
        *bytes = qk_workspace(a);
        return MU_OK;
    });
}

int mu_qk_max_logits(const mu_qk_logits* a, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check(a);
        if (rc) return rc;
        const bool empty = a->batch == 0 || a->q_len == 0 || a->k_len == 0;
        if (empty && a->accumulate) return MU_OK;
        const size_t need = qk_workspace(a);
        if (need) {
            if (!ws) return fail(MU_ERR_WORKSPACE, "workspace is null (need %zu bytes)", need);
            if (!aligned(ws, ALIGN)) return fail(MU_ERR_WORKSPACE, "workspace must be 256-byte aligned");
            if (ws_bytes < need) return fail(MU_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
        }
        const int es = a->dtype == MU_BF16 ? 2 : 4;
        // rows as whole 16-byte chunks, a tile of them within 32-bit offsets
        const int64_t mix = a->q_stride_b | a->q_stride_s | a->q_stride_h | a->k_stride_b | a->k_stride_s | a->k_stride_h | a->dim;
        const bool direct = (mix * es) % 16 == 0 && aligned(a->q, 16) && aligned(a->k, 16) &&
                            a->k_stride_s < ((int64_t)1 << 30) / (64 * es);
        // the profiler's figures (lengths on the device: operations unknown, bytes of all rows)
        const double nb = a->cu_q ? 1 : a->batch, nq = (double)a->q_len, nk = (double)a->k_len;
        const double bytes = nb * a->dim * es * (nq * a->q_heads + nk * a->k_heads);
        const double flops = a->cu_q || a->q_lengths || a->k_lengths ? 0.0 : 2.0 * nb * visible_pairs(nq, nk, a->causal) * a->q_heads * a->dim;
        return run_any(Call{a, (int64_t*)ws, direct, flops, bytes, (hipStream_t)stream});
    });
}

}  // extern "C"
