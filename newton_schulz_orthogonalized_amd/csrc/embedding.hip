// Embedding lookup and its gradient (gfx950): the C entry points and their
// kernels.
//
//   out[t, :]  = scale * weight[tokens[t], :]
//   grad[v, :] = scale * sum over t with tokens[t] == v, in rising t, of rows[t, :]
//
// The gradient sorts the tokens (stable, by least significant digits; tokens
// outside the table and the padding token sort behind all others), then sums
// the rows in sorted order: chunks of C consecutive entries, a wave for each
// chunk and slice of columns, whatever the distribution of the tokens. A run
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
// output written.
// ---------------------------------------------------------------------------
constexpr int TOK = 4;
struct LookupArgs {
    mu_lookup e;
    int lanes, slices;
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
        if (whole) *(MU_GLOBAL VU*)(o + j * E.dim) = v[j];
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
constexpr int STHR = 1024, SWAVES = STHR / 64;
constexpr int DIGIT = 9, RADIX = 1 << DIGIT;      // two passes up to 2^18 - 1 rows
constexpr int SORT_ONE = 16384;                   // tokens that one workgroup sorts by itself
constexpr int SORT_TILE = 8192;                   // tokens of a workgroup otherwise

struct SortArgs {
    mu_rowgrad e;
    const int32_t* key_in;   // null in the first pass: keys are made from the tokens
    const int32_t* pos_in;
    int32_t* key_out;
    int32_t* pos_out;
    int32_t* hist;           // [RADIX][tiles] digit counts of each tile
    int n, tiles;
    int shift;               // digit of this pass
    int passes;              // one-workgroup sort: all of them
    // the gradient's zeros are written by further workgroups of the sorting launches
    char* fill;
    int64_t fill_bytes;
    int sorters;             // workgroups 0 .. sorters - 1 sort
};

// Zeros, FILL_WG bytes a workgroup: sorting keeps one or a few compute units
// busy and waits on latency, so it runs beside the stores rather than before.
constexpr int64_t FILL_WG = (int64_t)STHR * 16 * 8;
__device__ __forceinline__ void fill_zeros(const SortArgs& A) {
    const int64_t at = (int64_t)(blockIdx.x - A.sorters) * FILL_WG;
    MU_GLOBAL char* p = (MU_GLOBAL char*)A.fill + at;
    const int64_t left = A.fill_bytes - at;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t o = ((int64_t)i * STHR + threadIdx.x) * 16;
        if (o + 16 <= left) *(MU_GLOBAL u32x4u*)(p + o) = u32x4{0, 0, 0, 0};
        else
            for (int64_t j = o; j < left; j += 2) *(MU_GLOBAL short*)(p + j) = 0;
    }
}

__device__ __forceinline__ uint32_t key_of(const SortArgs& A, int t) {
    const int64_t v = token_at(A.e.tokens, A.e.token_bits, t);
    return v >= 0 && v < A.e.vocab && v != A.e.padding_idx ? (uint32_t)v : (uint32_t)A.e.vocab;
}

// Stable rank of each lane's digit among those of its wave, counted on in
// cnt[digit]; lanes with the same digit find each other by one ballot a bit.
__device__ __forceinline__ int wave_rank(uint32_t d, bool on, volatile LDSP int* cnt) {
    uint64_t same = __ballot(on);
#pragma unroll
    for (int b = 0; b < DIGIT; ++b) {
        const bool bit = (d >> b) & 1;
        const uint64_t m = __ballot(on && bit);
        same &= bit ? m : ~m;
    }
    const int lane = threadIdx.x & 63;
    const int below = __popcll(same & ((1ull << lane) - 1));
    int base = 0;
    if (on) base = cnt[d];
    // (a wave's LDS accesses keep their order: every read above comes first)
    if (on && below == 0) cnt[d] = base + __popcll(same);
    return base + below;
}

// Exclusive sum over the workgroup in thread order.
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
    for (int i = 0; i < SWAVES; ++i)
        if (i < w) before += wsum[i];
    __syncthreads();
    return before;
}

// Up to SORT_ONE tokens in one workgroup: item i * 64 + lane of wave w's run of
// ipt * 64 items is thread (w, lane)'s i-th, so that rising (w, i, lane) is the
// items' order and ranks taken in it are stable. All passes stay in LDS.
// About 12 us for 8192 tokens and two passes, beside the stores of the zeros.
__global__ __launch_bounds__(STHR) void k_sort_one(SortArgs A) {
    __shared__ uint32_t skey[SORT_ONE];
    __shared__ uint16_t spos[SORT_ONE];
    __shared__ int cnt[SWAVES * RADIX];
    __shared__ int wsum[SWAVES];
    if ((int)blockIdx.x >= A.sorters) {
        fill_zeros(A);
        return;
    }
    constexpr int IPT = SORT_ONE / STHR;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int ipt = (A.n + STHR - 1) / STHR, first = w * ipt * 64 + lane;
    uint32_t key[IPT];
    int pos[IPT], rank[IPT];
    // behind the items: keys that sort last
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        pos[i] = first + i * 64;
        key[i] = i < ipt && pos[i] < A.n ? key_of(A, pos[i]) : 0xffffffffu;
    }
    for (int pass = 0; pass < A.passes; ++pass) {
        for (int i = tid; i < SWAVES * RADIX; i += STHR) cnt[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < IPT; ++i)
            if (i < ipt) rank[i] = wave_rank((key[i] >> (pass * DIGIT)) & (RADIX - 1), true, (volatile LDSP int*)cnt + w * RADIX);
        __syncthreads();
        // cnt[w][d] -> items of smaller digits, and of this digit in earlier waves
        {
            const int d = tid >> 1, w0 = (tid & 1) * (SWAVES / 2);
            int c[SWAVES / 2], sum = 0;
#pragma unroll
            for (int k = 0; k < SWAVES / 2; ++k) {
                c[k] = cnt[(w0 + k) * RADIX + d];
                sum += c[k];
            }
            int before = block_scan(sum, wsum);
#pragma unroll
            for (int k = 0; k < SWAVES / 2; ++k) {
                cnt[(w0 + k) * RADIX + d] = before;
                before += c[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < IPT; ++i)
            if (i < ipt) {
                const int to = cnt[w * RADIX + ((key[i] >> (pass * DIGIT)) & (RADIX - 1))] + rank[i];
                skey[to] = key[i];
                spos[to] = (uint16_t)pos[i];
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < IPT; ++i)
            if (i < ipt) {
                key[i] = skey[first + i * 64];
                pos[i] = spos[first + i * 64];
            }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = first + i * 64;
        if (i < ipt && j < A.n) {
            gp(A.key_out)[j] = (int32_t)key[i];
            gp(A.pos_out)[j] = pos[i];
        }
    }
}
static_assert(RADIX * 2 == STHR, "two threads a digit");

// More tokens: two launches a pass over tiles of SORT_TILE.
constexpr int TIPT = SORT_TILE / STHR;
__device__ __forceinline__ void tile_items(const SortArgs& A, uint32_t key[TIPT], int pos[TIPT], bool on[TIPT]) {
    const int first = blockIdx.x * SORT_TILE + (threadIdx.x >> 6) * TIPT * 64 + (threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < TIPT; ++i) {
        const int j = first + i * 64;
        on[i] = j < A.n;
        key[i] = !on[i] ? 0 : A.key_in ? (uint32_t)gp(A.key_in)[j] : key_of(A, j);
        pos[i] = !on[i] ? 0 : A.key_in ? gp(A.pos_in)[j] : j;
    }
}

__global__ __launch_bounds__(STHR) void k_sort_count(SortArgs A) {
    __shared__ int cnt[RADIX];
    if ((int)blockIdx.x >= A.sorters) {
        fill_zeros(A);
        return;
    }
    for (int i = threadIdx.x; i < RADIX; i += STHR) cnt[i] = 0;
    uint32_t key[TIPT];
    int pos[TIPT];
    bool on[TIPT];
    tile_items(A, key, pos, on);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TIPT; ++i)
        if (on[i]) atomicAdd(&cnt[(key[i] >> A.shift) & (RADIX - 1)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < RADIX; i += STHR) gp(A.hist)[(int64_t)i * A.tiles + blockIdx.x] = cnt[i];
}

__global__ __launch_bounds__(STHR) void k_sort_place(SortArgs A) {
    __shared__ int cnt[SWAVES * RADIX];
    __shared__ int wsum[SWAVES];
    if ((int)blockIdx.x >= A.sorters) {
        fill_zeros(A);
        return;
    }
    const int tid = threadIdx.x, w = tid >> 6;
    for (int i = tid; i < SWAVES * RADIX; i += STHR) cnt[i] = 0;
    uint32_t key[TIPT];
    int pos[TIPT], rank[TIPT];
    bool on[TIPT];
    tile_items(A, key, pos, on);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TIPT; ++i) rank[i] = wave_rank((key[i] >> A.shift) & (RADIX - 1), on[i], (volatile LDSP int*)cnt + w * RADIX);
    // where this tile's items of digit d go: behind all smaller digits, and
    // behind digit d of the tiles before
    int all = 0, mine = 0;
    if (tid < RADIX)
        for (int t = 0; t < A.tiles; ++t) {
            const int c = gp(A.hist)[(int64_t)tid * A.tiles + t];
            all += c;
            if (t < (int)blockIdx.x) mine += c;
        }
    const int to0 = block_scan(all, wsum) + mine;
    if (tid < RADIX) {
        int before = to0;
        for (int k = 0; k < SWAVES; ++k) {
            const int c = cnt[k * RADIX + tid];
            cnt[k * RADIX + tid] = before;
            before += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TIPT; ++i)
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
template <typename TR, typename TG>
__global__ __launch_bounds__(NTHR_SUM) void k_sum_rows(SumArgs A) {
    constexpr int U = 8;   // rows in flight
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
    uint32_t cur = (uint32_t)key[i0];
    if (cur >= vocab) return;
    bool from_before = i0 > 0 && (uint32_t)key[i0 - 1] == cur;
    const uint32_t behind = i1 < A.n ? (uint32_t)key[i1] : 0xffffffffu;
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    MU_GLOBAL float* part = (MU_GLOBAL float*)A.part + c * 2 * A.e.dim + col;
    auto flush = [&](bool goes_on) {
        if (from_before) store8<float>(part, cnt, s);
        else if (goes_on) store8<float>(part + A.e.dim, cnt, s);
        else put_row<TG>(A, cur, col, cnt, s);
    };
    for (int i = i0; i < i1; i += U) {
        uint32_t k[U];
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            k[u] = i + u < i1 ? (uint32_t)key[i + u] : 0xffffffffu;
            if (k[u] < vocab) load8<TR>(rows + (int64_t)pos[i + u] * A.e.dim, cnt, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k[u] >= vocab) continue;
            if (k[u] != cur) {
                flush(false);
                cur = k[u];
                from_before = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += v[u][e];
        }
    }
    flush(cur == behind);
}

// Joins the partial sums of the runs that cross chunk borders: a workgroup for
// the chunk in which the run starts and a slice of 64 lanes' columns; its four
// waves take a quarter of a long run's partials each and add up in order.
template <typename TG>
__global__ __launch_bounds__(NTHR_SUM) void k_join(SumArgs A) {
    __shared__ float q[3][64][8];
    const int c = blockIdx.x, i0 = c * A.chunk, i1 = i0 + A.chunk;
    if (i1 >= A.n) return;
    const MU_GLOBAL int32_t* key = (const MU_GLOBAL int32_t*)A.key;
    const uint32_t cur = (uint32_t)key[i1 - 1];
    if (cur >= (uint32_t)A.e.vocab || (uint32_t)key[i1] != cur) return;   // nothing goes on
    if ((uint32_t)key[i0] == cur && i0 > 0 && (uint32_t)key[i0 - 1] == cur) return;   // started before
    // chunks c + 1 .. end hold more of it: doubling steps, then halving
    int lo = c + 1, step = 1;   // the run reaches chunk lo
    while (lo + step < A.chunks && (uint32_t)key[(int64_t)(lo + step) * A.chunk] == cur) lo += step, step *= 2;
    for (; step >= 1; step /= 2)
        if (lo + step < A.chunks && (uint32_t)key[(int64_t)(lo + step) * A.chunk] == cur) lo += step;
    const int n = lo - c;   // partials behind the first
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
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
    if (e->accumulate != 0 && e->accumulate != 1) return fail(MU_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (e->padding_idx < -1 || e->padding_idx >= e->vocab)
        return fail(MU_ERR_INVALID_ARG, "padding_idx must be -1 or in [0, vocab)");
    return MU_OK;
}

// What a call of these sizes launches and keeps in its workspace.
struct GradPlan {
    int n, passes, tiles, chunk, chunks, lanes, slices;
    size_t off_key[2], off_pos[2], off_hist, off_part, bytes;
};
GradPlan grad_plan(const mu_rowgrad* e) {
    GradPlan p;
    p.n = (int)e->n_tokens;
    int bits = 1;
    while (bits < 32 && (e->vocab >> bits) != 0) ++bits;   // keys 0 .. vocab
    p.passes = (bits + DIGIT - 1) / DIGIT;
    p.tiles = p.n <= SORT_ONE ? 1 : (p.n + SORT_TILE - 1) / SORT_TILE;
    // short chunks while tokens are few (more waves), longer ones as their
    // partial sums would pass 64 MB
    p.chunk = 16;
    while (p.chunk < 1024 && 8.0 * (double)e->dim * (p.n / p.chunk) > (double)(64 << 20)) p.chunk *= 2;
    p.chunks = (p.n + p.chunk - 1) / p.chunk;
    p.lanes = 64;
    while (p.lanes > 1 && (int64_t)p.lanes / 2 * 8 >= e->dim) p.lanes /= 2;
    p.slices = (int)((e->dim + (int64_t)p.lanes * 8 - 1) / (p.lanes * 8));
    size_t o = 0;
    auto take = [&](size_t n) {
        const size_t at = o;
        o = align_up(o + n);
        return at;
    };
    for (int k = 0; k < 2; ++k) {
        const size_t n = k == 0 || p.tiles > 1 ? sizeof(int32_t) * (size_t)p.n : 0;
        p.off_key[k] = take(n);
        p.off_pos[k] = take(n);
    }
    p.off_hist = take(p.tiles > 1 ? sizeof(int32_t) * RADIX * (size_t)p.tiles : 0);
    p.off_part = take(p.chunks > 1 ? sizeof(float) * 2 * (size_t)p.chunks * (size_t)e->dim : 0);
    p.bytes = o;
    return p;
}

template <typename TR, typename TG>
hipError_t launch_sum(const SumArgs& a, hipStream_t s) {
    const int64_t groups = (int64_t)a.chunks * a.slices, per = NTHR_SUM / a.lanes;
    hipLaunchKernelGGL((k_sum_rows<TR, TG>), dim3((unsigned)((groups + per - 1) / per)), dim3(NTHR_SUM), 0, s, a);
    return hipGetLastError();
}

int run_rowgrad(const mu_rowgrad* e, char* ws, hipStream_t s) {
    const GradPlan p = grad_plan(e);
    const size_t er = es_of(e->row_dtype), eg = es_of(e->grad_dtype);
    // zeros in equal shares of the sorting launches (a multiple of 16 bytes each)
    const int64_t zeros = e->accumulate ? 0 : e->vocab * e->dim * (int64_t)eg;
    const int launches = p.n == 0 ? 1 : p.tiles == 1 ? 1 : 2 * p.passes;
    const int64_t share = (zeros / launches + 15) / 16 * 16;
    int done = 0;
    auto sort_launch = [&](void (*kernel)(SortArgs), SortArgs a, int sorters, double bytes) {
        const int64_t from = std::min(zeros, share * done), to = done + 1 == launches ? zeros : std::min(zeros, share * (done + 1));
        ++done;
        a.fill = (char*)e->grad + from;
        a.fill_bytes = to - from;
        a.sorters = sorters;
        const int64_t grid = sorters + (a.fill_bytes + FILL_WG - 1) / FILL_WG;
        if (grid == 0) return (int)MU_OK;
        return timed_launch(MU_K_ROWGRAD, 0.0, bytes + (double)a.fill_bytes, s, [&] {
            hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(STHR), 0, s, a);
            return hipGetLastError();
        }, "embedding gradient sort launch");
    };
    SortArgs a{};
    a.e = *e;
    a.n = p.n;
    a.tiles = p.tiles;
    a.passes = p.passes;
    a.hist = (int32_t*)(ws + p.off_hist);
    int out = 0;   // the buffer that holds the sorted keys at the end
    if (p.tiles == 1) {
        a.key_out = (int32_t*)(ws + p.off_key[0]);
        a.pos_out = (int32_t*)(ws + p.off_pos[0]);
        const int rc = sort_launch(k_sort_one, a, p.n > 0 ? 1 : 0, (double)p.n * (e->token_bits / 8 + 8));
        if (rc) return rc;
    } else {
        for (int k = 0; k < p.passes; ++k) {
            a.shift = k * DIGIT;
            a.key_in = k == 0 ? nullptr : (const int32_t*)(ws + p.off_key[out ^ 1]);
            a.pos_in = k == 0 ? nullptr : (const int32_t*)(ws + p.off_pos[out ^ 1]);
            a.key_out = (int32_t*)(ws + p.off_key[out]);
            a.pos_out = (int32_t*)(ws + p.off_pos[out]);
            int rc = sort_launch(k_sort_count, a, p.tiles, 8.0 * p.n);
            if (rc) return rc;
            rc = sort_launch(k_sort_place, a, p.tiles, 16.0 * p.n);
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
    const double row = (double)p.n * e->dim;
    int rc = timed_launch(MU_K_ROWGRAD, row, row * (er + eg), s, [&] {
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
        return timed_launch(MU_K_LOOKUP, 0.0, bytes, s, [&] {
            LookupArgs a{*e, 64, 0};
            const int epv = (int)(16 / es);
            while (a.lanes > 1 && (int64_t)a.lanes / 2 * epv >= e->dim) a.lanes /= 2;
            a.slices = (int)((e->dim + (int64_t)a.lanes * epv - 1) / (a.lanes * epv));
            const int64_t groups = (e->n_tokens + TOK - 1) / TOK * a.slices, per = NTHR / a.lanes;
            const dim3 grid((unsigned)((groups + per - 1) / per)), block(NTHR);
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
