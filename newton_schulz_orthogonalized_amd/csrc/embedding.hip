// Embedding lookup and its gradient (gfx950): the C entry points and their
// kernels.
//
//   out[t, :]  = scale * weight[tokens[t], :]
//   grad[v, :] = scale * sum over t with tokens[t] == v, in rising t, of rows[t, :]
//
// The gradient sorts the tokens (stable; tokens outside the table and the
// padding token sort behind all others), then sums the rows in sorted order:
// chunks of consecutive entries, a wave for each chunk and slice of columns,
// whatever the distribution of the tokens. A run
// of equal tokens inside a chunk is a finished row; a run that crosses chunk
// borders leaves a float32 partial sum in each chunk, and a last launch joins
// them in order. Every sum's order is fixed by the tokens.
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

__device__ __forceinline__ int64_t token_at(const void* tokens, int bits, int64_t t) {
    return bits == 32 ? (int64_t)((const MU_GLOBAL int32_t*)tokens)[t] : ((const MU_GLOBAL int64_t*)tokens)[t];
}

// Vectors at element alignment: gfx950 takes global vector accesses at any address.
typedef bf16x8 bf16x8u __attribute__((aligned(2)));
typedef f32x4 f32x4u __attribute__((aligned(4)));
typedef u32x4 u32x4u __attribute__((aligned(2)));

// Elements 0 .. cnt - 1 of eight as float32, zeros behind them.
template <typename T>
__device__ __forceinline__ void load8(const MU_GLOBAL T* p, int cnt, float v[8]) {
    if (cnt >= 8) {
        if constexpr (sizeof(T) == 2) {
            const bf16x8 q = *(const MU_GLOBAL bf16x8u*)p;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)q[e];
        } else {
            const f32x4 a = *(const MU_GLOBAL f32x4u*)p, b = *(const MU_GLOBAL f32x4u*)(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[e + 4] = b[e]; }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < cnt ? to_f32<T>(p[e]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(MU_GLOBAL T* p, int cnt, const float v[8]) {
    if (cnt >= 8) {
        if constexpr (sizeof(T) == 2) {
            bf16x8 q;
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = (bf16)v[e];
            *(MU_GLOBAL bf16x8u*)p = q;
        } else {
            *(MU_GLOBAL f32x4u*)p = f32x4{v[0], v[1], v[2], v[3]};
            *(MU_GLOBAL f32x4u*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    } else {
        for (int e = 0; e < cnt; ++e) p[e] = from_f32<T>(v[e]);
    }
}

// ---------------------------------------------------------------------------
// Lookup. A group of `lanes` lanes copies one 16-byte piece a lane of TOK rows,
// all loads before the first store. Bound by memory: the rows read once and the
// output written (16384 rows of 8 KB: 33 us, 191 MB at 5.7 TB/s; 8 rows a group, or
// loads that go past the caches, took 3 to 4 us more).
//
// Outputs of PAST_CACHES (half the last-level cache) and more are written past the
// caches: from there on what reads them next gains too, or loses little. Past them
// and not, in us, alone / with a norm / an elementwise product / a matrix product
// that reads them next (rows of 8 KB, a batch and an output of 3 GB in turn, as a
// training loop comes back to an output only after a whole step): 64 MB 21 and 24 /
// 38 and 39 / 48 and 45 / 87 and 85; 96 MB 30 and 33 / 52 and 53 / 67 and 65 / 118
// and 115; 128 MB 39 and 42 / 65 and 65 / 87 and 87 / 149 and 145; 160 MB 48 and 51 /
// 79 and 81 / 107 and 107 / 200 and 195; 192 MB 57 and 60 / 92 and 93 / 126 and 128 /
// 230 and 226; 256 MB 75 and 78 / 120 and 136 / 164 and 171 / 291 and 289; 512 MB 146
// and 149 / 228 and 229 / 317 and 328 / 573 and 574.
// ---------------------------------------------------------------------------
constexpr double PAST_CACHES = 128 << 20;
constexpr int TOK = 4;
struct LookupArgs {
    mu_lookup e;
    int lanes, slices;
    bool large;   // output written past the caches
};
template <typename T, bool SCALED>
__global__ __launch_bounds__(NTHR) void k_lookup(LookupArgs A) {
    constexpr int EPV = 16 / (int)sizeof(T);
    typedef T V __attribute__((ext_vector_type(EPV)));
    typedef V VU __attribute__((aligned(sizeof(T))));
    const mu_lookup& E = A.e;
    const int64_t g = ((int64_t)blockIdx.x * NTHR + threadIdx.x) / A.lanes;
    const int64_t t0 = g / A.slices * TOK;
    const int64_t col = ((g % A.slices) * A.lanes + threadIdx.x % A.lanes) * EPV;
    if (t0 >= E.n_tokens || col >= E.dim) return;
    const bool whole = col + EPV <= E.dim;
    const MU_GLOBAL T* w = (const MU_GLOBAL T*)E.weight + col;
    MU_GLOBAL T* o = (MU_GLOBAL T*)E.out + t0 * E.dim + col;
    const int n = (int)min<int64_t>(TOK, E.n_tokens - t0);
    V v[TOK];
    int64_t id[TOK];
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        id[j] = j < n ? token_at(E.tokens, E.token_bits, t0 + j) : -1;
        if (id[j] < 0 || id[j] >= E.vocab) {
            // a token outside the table reads nothing
#pragma unroll
            for (int e = 0; e < EPV; ++e) v[j][e] = (T)__builtin_nanf("");
            continue;
        }
        const MU_GLOBAL T* r = w + id[j] * E.dim;
        if (whole) v[j] = *(const MU_GLOBAL VU*)r;
        else {
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                if (col + e < E.dim) v[j][e] = r[e];
        }
    }
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        if (j >= n) break;
        if constexpr (SCALED) {
#pragma unroll
            for (int e = 0; e < EPV; ++e) v[j][e] = from_f32<T>(E.scale * to_f32<T>(v[j][e]));
        }
        if (whole && A.large) __builtin_nontemporal_store(v[j], (MU_GLOBAL VU*)(o + j * E.dim));
        else if (whole) *(MU_GLOBAL VU*)(o + j * E.dim) = v[j];
        else {
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                if (col + e < E.dim) o[j * E.dim + e] = v[j][e];
        }
    }
}

// ---------------------------------------------------------------------------
// Sort. Keys are table rows, `vocab` for tokens that add nothing.
// ---------------------------------------------------------------------------
constexpr int DIGIT = 9, RADIX = 1 << DIGIT;      // two passes up to 2^18 - 1 rows
constexpr int SORT_IPT = 8;                       // digit passes: tokens a thread

struct SortArgs {
    mu_rowgrad e;
    const int32_t* key_in;   // null in the first pass: keys are made from the tokens
    const int32_t* pos_in;
    int32_t* key_out;
    int32_t* pos_out;
    int32_t* hist;           // [RADIX][tiles] digit counts of each tile
    int32_t* totals;         // [RADIX] of each digit; null while every tile adds up all counts
    int n, tiles;
    int shift;               // digit of this pass
    int index_bits;          // counting: bits of a token's place
    // the gradient's zeros are written by further workgroups of the sorting launches
    char* fill;
    int64_t fill_bytes;
    int sorters;             // workgroups 0 .. sorters - 1 sort
};

// Zeros, FILL_WG bytes a workgroup: the sort computes and waits on latency, so
// it runs beside the stores rather than before.
constexpr int64_t FILL_WG = 65536;
__device__ __forceinline__ void fill_zeros(const SortArgs& A) {
    // one contiguous run of memory for each XCD
    const int64_t at = (int64_t)xcd_remap(blockIdx.x - A.sorters, gridDim.x - A.sorters) * FILL_WG;
    if (at >= A.fill_bytes) return;
    MU_GLOBAL char* p = (MU_GLOBAL char*)A.fill + at;
    const int64_t left = min<int64_t>(FILL_WG, A.fill_bytes - at);
    const int step = (int)blockDim.x * 16;
    if (left == FILL_WG) {
#pragma unroll 8
        for (int o = (int)threadIdx.x * 16; o < (int)FILL_WG; o += step) *(MU_GLOBAL u32x4u*)(p + o) = u32x4{0, 0, 0, 0};
        return;
    }
    for (int64_t o = (int64_t)threadIdx.x * 16; o < left; o += step) {
        if (o + 16 <= left) *(MU_GLOBAL u32x4u*)(p + o) = u32x4{0, 0, 0, 0};
        else
            for (int64_t j = o; j < left; j += 2) *(MU_GLOBAL short*)(p + j) = 0;
    }
}

__device__ __forceinline__ uint32_t key_of(const SortArgs& A, int t) {
    const int64_t v = token_at(A.e.tokens, A.e.token_bits, t);
    return v >= 0 && v < A.e.vocab && v != A.e.padding_idx ? (uint32_t)v : (uint32_t)A.e.vocab;
}

// Few tokens: a token's place is the number of tokens that sort before it. With
// key and place in one word (the place below the key) these are the smaller
// words. A workgroup holds all words in LDS and places RANK_ITEMS tokens; a lane
// compares RANK_LANE of them with one of RANK_PARTS runs of words, so that a
// word read from LDS serves four comparisons. n^2 comparisons spread over the
// chip, one launch and no passes: 8192 tokens 11 us (256 threads a workgroup
// 17.4, 512 13.1: one wave a SIMD does not hide its own latencies), bound by the
// comparisons (2.5 operations each) and by every workgroup reading every token;
// digit passes of one workgroup took 22 us, of small tiles about 25.
constexpr int RANK_THR = 1024, RANK_ITEMS = 32, RANK_LANE = 4, RANK_PARTS = RANK_THR / (RANK_ITEMS / RANK_LANE);
template <typename W>
__global__ __launch_bounds__(RANK_THR) void k_sort_rank(SortArgs A) {
    extern __shared__ __align__(16) char raw[];
    __shared__ int count[RANK_THR / 64][RANK_ITEMS];
    if ((int)blockIdx.x >= A.sorters) {
        fill_zeros(A);
        return;
    }
    constexpr int PER = 16 / (int)sizeof(W);   // words of one LDS read
    typedef W WV __attribute__((ext_vector_type(PER)));
    LDSP W* word = (LDSP W*)(LDSP char*)raw;
    const int tid = threadIdx.x;
    // run q is reads q, q + RANK_PARTS, ..: the runs of a wave read side by side
    const int reads = (A.n + PER * RANK_PARTS - 1) / (PER * RANK_PARTS) * RANK_PARTS, words = reads * PER;
    // (each workgroup begins elsewhere: all at one place would queue at one
    // memory channel)
    const int start = (int)((int64_t)words * (blockIdx.x >> 3) / ((A.sorters >> 3) + 1)) / RANK_THR * RANK_THR;
#pragma unroll 16
    for (int j = tid; j < words; j += RANK_THR) {
        int i = j + start;
        if (i >= words) i -= words;
        word[i] = i < A.n ? ((W)key_of(A, min(i, A.n - 1)) << A.index_bits) | (W)i : ~(W)0 >> 1;
    }
    __syncthreads();
    const int g = tid % (RANK_ITEMS / RANK_LANE), q = tid / (RANK_ITEMS / RANK_LANE), first = blockIdx.x * RANK_ITEMS;
    W mine[RANK_LANE];
    int n[RANK_LANE];
#pragma unroll
    for (int k = 0; k < RANK_LANE; ++k) {
        mine[k] = word[min(first + g * RANK_LANE + k, A.n - 1)];
        n[k] = 0;
    }
#pragma unroll 4
    for (int i = q; i < reads; i += RANK_PARTS) {
        const WV x = ((const LDSP WV*)word)[i];
#pragma unroll
        for (int k = 0; k < RANK_LANE; ++k)
#pragma unroll
            for (int e = 0; e < PER; ++e) n[k] += (int)((x[e] - mine[k]) >> (8 * sizeof(W) - 1));   // 1 where x < mine
    }
#pragma unroll
    for (int k = 0; k < RANK_LANE; ++k) {
        for (int off = RANK_ITEMS / RANK_LANE; off < 64; off *= 2) n[k] += __shfl_xor(n[k], off, 64);
        if ((tid & 63) == g) count[tid >> 6][g * RANK_LANE + k] = n[k];
    }
    __syncthreads();
    const int item = first + tid;
    if (tid >= RANK_ITEMS || item >= A.n) return;
    int to = 0;
#pragma unroll
    for (int k = 0; k < RANK_THR / 64; ++k) to += count[k][tid];
    gp(A.key_out)[to] = (int32_t)(word[item] >> A.index_bits);
    gp(A.pos_out)[to] = item;
}

// More tokens: two launches for each digit, over tiles of THR * SORT_IPT.
//
// Stable rank of each lane's digit among those of its wave, counted on in
// cnt[digit]; lanes with the same digit find each other by one ballot a bit.
__device__ __forceinline__ int wave_rank(uint32_t d, bool on, volatile LDSP int* cnt) {
    const uint64_t all = __ballot(on);
    uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
#pragma unroll
    for (int b = 0; b < DIGIT; ++b) {
        const uint32_t bit = (uint32_t)((int32_t)(d << (31 - b)) >> 31);   // all ones where set
        const uint64_t m = __ballot(bit != 0);
        lo &= ~((uint32_t)m ^ bit);
        hi &= ~((uint32_t)(m >> 32) ^ bit);
    }
    const int below = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
    int base = 0;
    if (on) base = cnt[d];
    // (a wave's LDS accesses keep their order: every read above comes first)
    if (on && below == 0) cnt[d] = base + __popc(lo) + __popc(hi);
    return base + below;
}

// Exclusive sum over the workgroup in thread order.
template <int THR>
__device__ __forceinline__ int block_scan(int v, int* wsum) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int s = v;
    for (int off = 1; off < 64; off <<= 1) {
        const int up = __shfl_up(s, off, 64);
        if (lane >= off) s += up;
    }
    if (lane == 63) wsum[w] = s;
    __syncthreads();
    int before = s - v;
#pragma unroll
    for (int i = 0; i < THR / 64; ++i)
        if (i < w) before += wsum[i];
    __syncthreads();
    return before;
}

// Thread (w, lane)'s i-th item is i * 64 + lane of wave w's run: rising (w, i,
// lane) is the items' order, and ranks taken in it are stable.
template <int THR>
__device__ __forceinline__ void tile_items(const SortArgs& A, uint32_t key[SORT_IPT], int pos[SORT_IPT], bool on[SORT_IPT]) {
    const int first = (int)blockIdx.x * (THR * SORT_IPT) + (int)(threadIdx.x >> 6) * SORT_IPT * 64 + (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < SORT_IPT; ++i) {
        const int j = min(first + i * 64, A.n - 1);
        on[i] = first + i * 64 < A.n;
        key[i] = A.key_in ? (uint32_t)gp(A.key_in)[j] : key_of(A, j);
        pos[i] = A.key_in ? gp(A.pos_in)[j] : j;
    }
}

template <int THR>
__global__ __launch_bounds__(THR) void k_sort_count(SortArgs A) {
    __shared__ int cnt[RADIX];
    if ((int)blockIdx.x >= A.sorters) {
        fill_zeros(A);
        return;
    }
    for (int i = threadIdx.x; i < RADIX; i += THR) cnt[i] = 0;
    uint32_t key[SORT_IPT];
    int pos[SORT_IPT];
    bool on[SORT_IPT];
    tile_items<THR>(A, key, pos, on);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_IPT; ++i)
        if (on[i]) atomicAdd(&cnt[(key[i] >> A.shift) & (RADIX - 1)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < RADIX; i += THR) gp(A.hist)[(int64_t)i * A.tiles + blockIdx.x] = cnt[i];
}

// Many tiles: a digit's counts become the items of the tiles before, one
// workgroup a digit.
constexpr int SCAN_THR = 256;
__global__ __launch_bounds__(SCAN_THR) void k_sort_scan(SortArgs A) {
    __shared__ int wsum[SCAN_THR / 64];
    __shared__ int last;
    MU_GLOBAL int32_t* h = gp(A.hist) + (int64_t)blockIdx.x * A.tiles;
    int carry = 0;
    for (int t0 = 0; t0 < A.tiles; t0 += SCAN_THR) {
        const int t = t0 + (int)threadIdx.x;
        const int c = t < A.tiles ? h[t] : 0;
        const int before = carry + block_scan<SCAN_THR>(c, wsum);
        if (t < A.tiles) h[t] = before;
        if (threadIdx.x == SCAN_THR - 1) last = before + c;
        __syncthreads();
        carry = last;
    }
    if (threadIdx.x == 0) gp(A.totals)[blockIdx.x] = carry;
}

template <int THR>
__global__ __launch_bounds__(THR) void k_sort_place(SortArgs A) {
    constexpr int WAVES = THR / 64, DPT = RADIX > THR ? RADIX / THR : 1;   // digits a thread adds up
    __shared__ int cnt[WAVES * RADIX];
    __shared__ int wsum[WAVES];
    if ((int)blockIdx.x >= A.sorters) {
        fill_zeros(A);
        return;
    }
    const int tid = threadIdx.x, w = tid >> 6;
    for (int i = tid; i < WAVES * RADIX; i += THR) cnt[i] = 0;
    uint32_t key[SORT_IPT];
    int pos[SORT_IPT], rank[SORT_IPT];
    bool on[SORT_IPT];
    tile_items<THR>(A, key, pos, on);
    // where this tile's items of digit d go: behind all smaller digits, and
    // behind digit d of the tiles before
    int all[DPT], mine[DPT], sum = 0;
#pragma unroll
    for (int k = 0; k < DPT; ++k) {
        all[k] = mine[k] = 0;
        const int d = tid * DPT + k;
        if (d < RADIX) {
            const MU_GLOBAL int32_t* h = gp(A.hist) + (int64_t)d * A.tiles;
            if (A.totals) {
                all[k] = gp(A.totals)[d];
                mine[k] = h[blockIdx.x];
            } else {
#pragma unroll 8
                for (int t = 0; t < A.tiles; ++t) {
                    const int c = h[t];
                    all[k] += c;
                    mine[k] += t < (int)blockIdx.x ? c : 0;
                }
            }
        }
        sum += all[k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_IPT; ++i)
        rank[i] = wave_rank((key[i] >> A.shift) & (RADIX - 1), on[i], (volatile LDSP int*)cnt + w * RADIX);
    int before = block_scan<THR>(sum, wsum);
#pragma unroll
    for (int k = 0; k < DPT; ++k) {
        const int d = tid * DPT + k;
        if (d < RADIX) {
            int to = before + mine[k];
            for (int i = 0; i < WAVES; ++i) {
                const int c = cnt[i * RADIX + d];
                cnt[i * RADIX + d] = to;
                to += c;
            }
        }
        before += all[k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_IPT; ++i)
        if (on[i]) {
            const int to = cnt[w * RADIX + ((key[i] >> A.shift) & (RADIX - 1))] + rank[i];
            gp(A.key_out)[to] = (int32_t)key[i];
            gp(A.pos_out)[to] = pos[i];
        }
}

// ---------------------------------------------------------------------------
// Sums of the sorted rows. A group of `lanes` lanes (a power of two, 64 at
// most) owns 8 columns a lane of one chunk.
// ---------------------------------------------------------------------------
struct SumArgs {
    mu_rowgrad e;
    const int32_t* key;
    const int32_t* pos;
    float* part;        // [chunks][2][dim]: a run that came from the chunk before; one that goes on behind
    int n, chunk, chunks;
    int lanes, slices;
};

template <typename TG>
__device__ __forceinline__ void put_row(const SumArgs& A, int64_t v, int64_t col, int cnt, const float s[8]) {
    MU_GLOBAL TG* g = (MU_GLOBAL TG*)A.e.grad + v * A.e.dim + col;
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = A.e.scale * s[k];
    if (A.e.accumulate) {
        float o[8];
        load8<TG>(g, cnt, o);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] += o[k];
    }
    store8<TG>(g, cnt, r);
}

constexpr int NTHR_SUM = 256;
// Eight columns of a row as they lie in memory. Rows are read once: non-temporal
// loads leave the zeros just written in the caches (the sums of the 8B-shaped
// gradient ran 36 -> 22 us, of the Llama-1B-shaped one 57 -> 41 us).
template <typename T> struct Raw8 {
    bf16x8 q;
    __device__ __forceinline__ void load(const MU_GLOBAL T* p) { q = __builtin_nontemporal_load((const MU_GLOBAL bf16x8u*)p); }
    __device__ __forceinline__ float operator[](int e) const { return (float)q[e]; }
    __device__ __forceinline__ void set(int e, T v) { q[e] = v; }
};
template <> struct Raw8<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const MU_GLOBAL float* p) {
        a = __builtin_nontemporal_load((const MU_GLOBAL f32x4u*)p);
        b = __builtin_nontemporal_load((const MU_GLOBAL f32x4u*)(p + 4));
    }
    __device__ __forceinline__ float operator[](int e) const { return e < 4 ? a[e] : b[e - 4]; }
    __device__ __forceinline__ void set(int e, float v) {
        if (e < 4) a[e] = v;
        else b[e - 4] = v;
    }
};
template <typename T>
__device__ __forceinline__ void load_raw(Raw8<T>& r, const MU_GLOBAL T* p, int cnt) {
    if (cnt >= 8) r.load(p);
    else
#pragma unroll
        for (int e = 0; e < 8; ++e) r.set(e, e < cnt ? p[e] : (T)0.f);
}

// SUM_U entries at a time: their keys and positions, then all their rows (ACC:
// and the gradient's rows that the runs ending there are added to) before the
// first addition. Bound by memory and, with few tokens, by its latency.
constexpr int SUM_U = 8;
template <typename TR, typename TG, bool ACC>
__global__ __launch_bounds__(NTHR_SUM) void k_sum_rows(SumArgs A) {
    const int64_t g = ((int64_t)blockIdx.x * NTHR_SUM + threadIdx.x) / A.lanes;
    const int64_t c = g / A.slices;
    if (c >= A.chunks) return;
    const int64_t col = ((g - c * A.slices) * A.lanes + threadIdx.x % A.lanes) * 8;
    const int cnt = (int)min<int64_t>(8, A.e.dim - col);
    if (cnt <= 0) return;
    const uint32_t vocab = (uint32_t)A.e.vocab;
    const int i0 = (int)c * A.chunk, i1 = min(A.n, i0 + A.chunk);
    const MU_GLOBAL int32_t* key = (const MU_GLOBAL int32_t*)A.key;
    const MU_GLOBAL int32_t* pos = (const MU_GLOBAL int32_t*)A.pos;
    const MU_GLOBAL TR* rows = (const MU_GLOBAL TR*)A.e.rows + col;
    MU_GLOBAL TG* grad = (MU_GLOBAL TG*)A.e.grad + col;
    MU_GLOBAL float* part = (MU_GLOBAL float*)A.part + c * 2 * A.e.dim + col;
    const float scale = A.e.scale;
    // keys of a batch and the one behind it; places past the chunk's end repeat
    // its last entry and are skipped
    uint32_t k[SUM_U + 1], kn[SUM_U + 1];
    int p[SUM_U];
    const uint32_t behind = i1 < A.n ? (uint32_t)key[i1] : 0xffffffffu;
    auto entries = [&](int i, uint32_t (&kk)[SUM_U + 1]) {
#pragma unroll
        for (int u = 0; u < SUM_U; ++u) {
            const int j = min(i + u, i1 - 1);
            kk[u] = (uint32_t)key[j];
            p[u] = pos[j];
        }
        kk[SUM_U] = i + SUM_U < i1 ? (uint32_t)key[i + SUM_U] : behind;
    };
    const uint32_t ahead = i0 > 0 ? (uint32_t)key[i0 - 1] : 0xffffffffu;
    entries(i0, k);
    if (k[0] >= vocab) return;
    bool from_before = ahead == k[0];
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    for (int i = i0; i < i1; i += SUM_U) {
        Raw8<TR> v[SUM_U];
        Raw8<TG> o[ACC ? SUM_U : 1];
        // (rows of tokens that add nothing are read too, and skipped)
#pragma unroll
        for (int u = 0; u < SUM_U; ++u) load_raw<TR>(v[u], rows + (int64_t)p[u] * A.e.dim, cnt);
        if constexpr (ACC) {
#pragma unroll
            for (int u = 0; u < SUM_U; ++u)
                if (k[u] < vocab && (u + 1 < SUM_U && i + u + 1 >= i1 ? behind : k[u + 1]) != k[u])
                    load_raw<TG>(o[u], grad + (int64_t)k[u] * A.e.dim, cnt);
        }
        entries(i + SUM_U, kn);
#pragma unroll
        for (int u = 0; u < SUM_U; ++u) {
            if (i + u >= i1 || k[u] >= vocab) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += v[u][e];
            const bool end = i + u + 1 >= i1;   // of the chunk
            const uint32_t next = end ? behind : k[u + 1];
            if (next == k[u] && !end) continue;
            // the run ends here, or goes on in the next chunk
            if (from_before) store8<float>(part, cnt, s);
            else if (next == k[u]) store8<float>(part + A.e.dim, cnt, s);
            else {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = scale * s[e];
                    if constexpr (ACC) x[e] += o[u][e];
                }
                store8<TG>(grad + (int64_t)k[u] * A.e.dim, cnt, x);
            }
            from_before = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = 0.f;
        }
#pragma unroll
        for (int u = 0; u <= SUM_U; ++u) k[u] = kn[u];
    }
}

// Joins the partial sums of the runs that cross chunk borders: a workgroup for
// the chunk in which the run starts and a slice of 64 lanes' columns; its four
// waves take a quarter of a long run's partials each and add up in order. (Most
// workgroups find nothing: with 16 waves each they cost 8192 chunks 33 us more.)
template <typename TG>
__global__ __launch_bounds__(NTHR_SUM) void k_join(SumArgs A) {
    __shared__ float q[3][64][8];
    const int c = blockIdx.x, i0 = c * A.chunk, i1 = i0 + A.chunk;
    if (i1 >= A.n) return;
    const MU_GLOBAL int32_t* key = (const MU_GLOBAL int32_t*)A.key;
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // asked for together: the border's keys, those of the chunk's begin, and
    // whether the run reaches each of the next 64 chunks
    int step = 1, lo = c;   // the run reaches chunk lo
    auto reached = [&] {   // of the chunks lo + step, lo + 2 step, ..
        const int64_t j = min<int64_t>(lo + (int64_t)(lane + 1) * step, A.chunks - 1) * A.chunk;
        return (uint32_t)key[j];
    };
    const uint32_t cur = (uint32_t)key[i1 - 1], next = (uint32_t)key[i1], begin = (uint32_t)key[i0];
    const uint32_t ahead = (uint32_t)key[max(i0 - 1, 0)];
    uint32_t at = reached();
    if (cur >= (uint32_t)A.e.vocab || next != cur) return;   // nothing goes on
    if (i0 > 0 && begin == cur && ahead == cur) return;      // started before
    // steps of 1, 64, .. chunks while all 64 are reached, then back to 1
    auto count = [&](uint32_t v) { return __popcll(__ballot(lo + (int64_t)(lane + 1) * step < A.chunks && v == cur)); };
    for (int m = count(at);; m = count(reached())) {
        lo += m * step;
        if (m < 64) break;
        step *= 64;
    }
    while (step > 1) {
        step /= 64;
        lo += count(reached()) * step;
    }
    const int n = lo - c;   // partials behind the first
    const int64_t col = ((int64_t)blockIdx.y * 64 + lane) * 8;
    const int cnt = (int)min<int64_t>(8, max<int64_t>(0, A.e.dim - col));
    const MU_GLOBAL float* part = (const MU_GLOBAL float*)A.part + col;
    const int per = n < 16 ? n : (n + 3) / 4, j0 = min(n, w * per), j1 = min(n, j0 + per);
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    if (w == 0 && cnt > 0) load8<float>(part + ((int64_t)c * 2 + 1) * A.e.dim, cnt, s);
    if (cnt > 0)
        for (int j = j0; j < j1; j += 8) {
            float v[8][8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j + u < j1) load8<float>(part + (int64_t)(c + 1 + j + u) * 2 * A.e.dim, cnt, v[u]);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j + u < j1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] += v[u][e];
                }
        }
    if (w > 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) q[w - 1][lane][e] = s[e];
    __syncthreads();
    if (w > 0 || cnt <= 0) return;
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += q[k][lane][e];
    put_row<TG>(A, cur, col, cnt, s);
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
    if (e->n_tokens > (1 << 30)) return fail(MU_ERR_INVALID_ARG, "n_tokens must be at most 2^30");
    if (e->accumulate != 0 && e->accumulate != 1) return fail(MU_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (e->padding_idx < -1 || e->padding_idx >= e->vocab)
        return fail(MU_ERR_INVALID_ARG, "padding_idx must be -1 or in [0, vocab)");
    return MU_OK;
}

// What a call of these sizes launches and keeps in its workspace.
struct GradPlan {
    int n, index_bits, word_bits, passes, thr, tiles, chunk, chunks, lanes, slices;
    bool scan;
    size_t off_key[2], off_pos[2], off_hist, off_totals, off_part, bytes;
};
// Tiles from which a launch of its own adds up their counts (each tile adding
// up all of them grows with the square): 64 tiles 67.2 us without and with,
// 128 tiles (262144 tokens) 137 and 129, 512 tiles 583 and 470.
constexpr int SCAN_TILES = 64;
// Waves of the sums from which chunks grow instead: fewer partial sums, shorter
// joins. 65536 x 4096 of which half are one token 440 us without a limit, 400,
// 373, 371 with 8192, 4096, 2048; 2^20 x 256 uniform 237, 203, 186, 190 and with
// half one token 711, 439, 308, 256; 2^21 x 64 343, 266, 209, 183.
constexpr int64_t WAVES_MAX = 2048;
GradPlan grad_plan(const mu_rowgrad* e) {
    GradPlan p;
    p.n = (int)e->n_tokens;
    int bits = 1;
    while (bits < 32 && (e->vocab >> bits) != 0) ++bits;   // keys 0 .. vocab
    p.passes = (bits + DIGIT - 1) / DIGIT;
    // small tiles while they are few, as more workgroups hide a tile's latencies:
    // 65536 tokens 49 us with 256 threads and 62 with 1024, 400000 101 and 114, but
    // 2^20 126 and 118, 2^22 332 and 298
    p.thr = p.n <= (1 << 19) ? 256 : 1024;
    // Counting or digit passes: 9000 tokens 33 against 46 us (768 columns), 12000
    // 39 against 48, 16384 51 against 48; with 64-bit words 32 against 34 at 9000
    // and 40 against 35 at 12000.
    p.index_bits = 0;
    while ((1 << p.index_bits) < p.n) ++p.index_bits;
    // words stay below half the type's range: the padding of the last reads is
    // above all, and a difference of two has the sign of its comparison
    p.word_bits = bits + p.index_bits < 31 ? 32 : 64;
    const bool rank = p.n <= (p.word_bits == 32 ? 12288 : 8192);
    p.tiles = rank ? 0 : (p.n + p.thr * SORT_IPT - 1) / (p.thr * SORT_IPT);
    p.scan = p.tiles > SCAN_TILES;
    p.lanes = 64;
    while (p.lanes > 1 && (int64_t)p.lanes / 2 * 8 >= e->dim) p.lanes /= 2;
    p.slices = (int)((e->dim + (int64_t)p.lanes * 8 - 1) / (p.lanes * 8));
    // short chunks while tokens are few (more waves)
    p.chunk = 16;
    while (p.chunk < 1024 && (int64_t)(p.n / p.chunk) * p.slices * p.lanes / 64 > WAVES_MAX) p.chunk *= 2;
    p.chunks = (p.n + p.chunk - 1) / p.chunk;
    size_t o = 0;
    auto take = [&](size_t n) {
        const size_t at = o;
        o = align_up(o + n);
        return at;
    };
    for (int k = 0; k < 2; ++k) {
        const size_t n = k == 0 || p.tiles > 0 ? sizeof(int32_t) * (size_t)p.n : 0;
        p.off_key[k] = take(n);
        p.off_pos[k] = take(n);
    }
    p.off_hist = take(p.tiles > 0 ? sizeof(int32_t) * RADIX * (size_t)p.tiles : 0);
    p.off_totals = take(p.scan ? sizeof(int32_t) * RADIX : 0);
    p.off_part = take(p.chunks > 1 ? sizeof(float) * 2 * (size_t)p.chunks * (size_t)e->dim : 0);
    p.bytes = o;
    return p;
}

template <typename TR, typename TG>
hipError_t launch_sum(const SumArgs& a, hipStream_t s) {
    const int64_t groups = (int64_t)a.chunks * a.slices, per = NTHR_SUM / a.lanes;
    const dim3 grid((unsigned)((groups + per - 1) / per));
    if (a.e.accumulate) hipLaunchKernelGGL((k_sum_rows<TR, TG, true>), grid, dim3(NTHR_SUM), 0, s, a);
    else hipLaunchKernelGGL((k_sum_rows<TR, TG, false>), grid, dim3(NTHR_SUM), 0, s, a);
    return hipGetLastError();
}

int run_rowgrad(const mu_rowgrad* e, char* ws, hipStream_t s) {
    const GradPlan p = grad_plan(e);
    const size_t er = es_of(e->row_dtype), eg = es_of(e->grad_dtype);
    // zeros in equal shares of the sorting launches (a multiple of 16 bytes each)
    const int64_t zeros = e->accumulate ? 0 : e->vocab * e->dim * (int64_t)eg;
    const int launches = p.tiles == 0 ? 1 : 2 * p.passes;
    const int64_t share = (zeros / launches + 15) / 16 * 16;
    int done = 0;
    auto sort_launch = [&](void (*kernel)(SortArgs), SortArgs a, int sorters, int thr, size_t lds, double bytes) {
        const int64_t from = std::min(zeros, share * done), to = done + 1 == launches ? zeros : std::min(zeros, share * (done + 1));
        ++done;
        a.fill = (char*)e->grad + from;
        a.fill_bytes = to - from;
        a.sorters = sorters;
        const int64_t grid = sorters + (a.fill_bytes + 8 * FILL_WG - 1) / (8 * FILL_WG) * 8;
        if (grid == 0) return (int)MU_OK;
        return timed_launch(MU_K_ROWGRAD, 0.0, bytes + (double)a.fill_bytes, s, [&] {
            hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(thr), lds, s, a);
            return hipGetLastError();
        }, "embedding gradient sort launch");
    };
    SortArgs a{};
    a.e = *e;
    a.n = p.n;
    a.tiles = p.tiles;
    a.hist = (int32_t*)(ws + p.off_hist);
    a.totals = p.scan ? (int32_t*)(ws + p.off_totals) : nullptr;
    int out = 0;   // the buffer that holds the sorted keys at the end
    if (p.tiles == 0) {
        a.key_out = (int32_t*)(ws + p.off_key[0]);
        a.pos_out = (int32_t*)(ws + p.off_pos[0]);
        a.index_bits = p.index_bits;
        const int groups = (p.n + RANK_ITEMS - 1) / RANK_ITEMS;
        const bool small = p.word_bits == 32;
        const int per = (small ? 4 : 2) * RANK_PARTS;   // words of one read of every run
        const size_t lds = (size_t)(p.n + per - 1) / per * 16 * RANK_PARTS;
        const int rc = sort_launch(small ? k_sort_rank<uint32_t> : k_sort_rank<uint64_t>, a, groups, RANK_THR, lds,
                                   (double)p.n * (e->token_bits / 8 + 8));
        if (rc) return rc;
    } else {
        for (int k = 0; k < p.passes; ++k) {
            a.shift = k * DIGIT;
            a.key_in = k == 0 ? nullptr : (const int32_t*)(ws + p.off_key[out ^ 1]);
            a.pos_in = k == 0 ? nullptr : (const int32_t*)(ws + p.off_pos[out ^ 1]);
            a.key_out = (int32_t*)(ws + p.off_key[out]);
            a.pos_out = (int32_t*)(ws + p.off_pos[out]);
            const bool few = p.thr == 256;
            int rc = sort_launch(few ? k_sort_count<256> : k_sort_count<1024>, a, p.tiles, p.thr, 0, 8.0 * p.n);
            if (rc) return rc;
            if (p.scan)
                rc = timed_launch(MU_K_ROWGRAD, 0.0, 8.0 * RADIX * p.tiles, s, [&] {
                    hipLaunchKernelGGL(k_sort_scan, dim3(RADIX), dim3(SCAN_THR), 0, s, a);
                    return hipGetLastError();
                }, "embedding gradient sort launch");
            if (rc) return rc;
            rc = sort_launch(few ? k_sort_place<256> : k_sort_place<1024>, a, p.tiles, p.thr, 0, 16.0 * p.n);
            if (rc) return rc;
            out ^= 1;
        }
        out ^= 1;
    }
    if (p.n == 0) return MU_OK;
    SumArgs b{};
    b.e = *e;
    b.key = (const int32_t*)(ws + p.off_key[out]);
    b.pos = (const int32_t*)(ws + p.off_pos[out]);
    b.part = (float*)(ws + p.off_part);
    b.n = p.n;
    b.chunk = p.chunk;
    b.chunks = p.chunks;
    b.lanes = p.lanes;
    b.slices = p.slices;
    // (tokens on the device: as if all were valid and as many rows named as can be;
    // the partial sums of runs that cross chunks are not counted)
    const double row = (double)p.n * e->dim, named = (double)std::min(e->n_tokens, e->vocab) * e->dim;
    int rc = timed_launch(MU_K_ROWGRAD, row, row * er + named * eg * (e->accumulate ? 2 : 1) + 8.0 * p.n, s, [&] {
        if (e->row_dtype == MU_BF16)
            return e->grad_dtype == MU_BF16 ? launch_sum<bf16, bf16>(b, s) : launch_sum<bf16, float>(b, s);
        return e->grad_dtype == MU_BF16 ? launch_sum<float, bf16>(b, s) : launch_sum<float, float>(b, s);
    }, "embedding gradient sum launch");
    if (rc || p.chunks == 1) return rc;
    return timed_launch(MU_K_ROWGRAD, 0.0, 0.0, s, [&] {
        const dim3 grid((unsigned)p.chunks, (unsigned)((e->dim + 511) / 512));
        if (e->grad_dtype == MU_BF16) hipLaunchKernelGGL(k_join<bf16>, grid, dim3(NTHR_SUM), 0, s, b);
        else hipLaunchKernelGGL(k_join<float>, grid, dim3(NTHR_SUM), 0, s, b);
        return hipGetLastError();
    }, "embedding gradient join launch");
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
        LookupArgs a{*e, 64, 0, (double)e->n_tokens * e->dim * es >= PAST_CACHES};
        const int epv = (int)(16 / es);
        while (a.lanes > 1 && (int64_t)a.lanes / 2 * epv >= e->dim) a.lanes /= 2;
        a.slices = (int)((e->dim + (int64_t)a.lanes * epv - 1) / (a.lanes * epv));
        const int64_t groups = (e->n_tokens + TOK - 1) / TOK * a.slices, per = NTHR / a.lanes, wgs = (groups + per - 1) / per;
        if (wgs > 0xffffffffLL / NTHR) return fail(MU_ERR_INVALID_ARG, "too many tokens for one launch at this dim");
        return timed_launch(MU_K_LOOKUP, 0.0, bytes, s, [&] {
            const dim3 grid((unsigned)wgs), block(NTHR);
            if (e->dtype == MU_BF16) {
                if (e->scale == 1.f) hipLaunchKernelGGL((k_lookup<bf16, false>), grid, block, 0, s, a);
                else hipLaunchKernelGGL((k_lookup<bf16, true>), grid, block, 0, s, a);
            } else {
                if (e->scale == 1.f) hipLaunchKernelGGL((k_lookup<float, false>), grid, block, 0, s, a);
                else hipLaunchKernelGGL((k_lookup<float, true>), grid, block, 0, s, a);
            }
            return hipGetLastError();
        }, "embedding launch");
    });
}

int mu_embedding_grad_workspace_size(const mu_rowgrad* e, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MU_ERR_INVALID_ARG, "bytes is null");
        int rc = check_rowgrad(e);
        if (rc) return rc;
        *bytes = grad_plan(e).bytes;
        return MU_OK;
    });
}

int mu_embedding_grad(const mu_rowgrad* e, void* ws, size_t ws_bytes, void* stream) {
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
        const size_t need = grad_plan(e).bytes;
        if (need) {
            if (!ws) return fail(MU_ERR_WORKSPACE, "workspace is null (need %zu bytes)", need);
            if (!aligned(ws, ALIGN)) return fail(MU_ERR_WORKSPACE, "workspace must be 256-byte aligned");
            if (ws_bytes < need) return fail(MU_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
        }
        return run_rowgrad(e, (char*)ws, (hipStream_t)stream);
    });
}

}  // extern "C"
