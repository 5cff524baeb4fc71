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
// What is rounded to bfloat16 on the way to its gradients: dg and du, where they leave
// k_slopes or RECOMP, because the matrix instructions that read them take bfloat16 (as two
// halves each they would be twice the work), and every result. Two roundings leave a
// gradient 0.0024 of its size off (2048 tokens of 4096 x 14336), one alone 0.0017. g and u
// are not: the forward call leaves them in float32, which costs 8192 tokens of 4096 x 14336
// 85 us forward (1435 -> 1520) and 110 in k_slopes against bfloat16. Those, which a caller
// may choose for half the memory, are a third rounding: 0.0030. (The same block in a
// library's bfloat16 operations, which round act(g) too: 0.0034 to 0.0039.)
//
// Slices of 128 bytes of k (64 bfloat16, 32 float32) move from memory to LDS with
// direct loads, 1 KB each; what lies outside an operand reads as zero.
//
// What bounds them: matrix instructions. Large bfloat16 products take the tiles of 256 of
// gated_wide.hip; here are those of 128 and 64 and all of float32, which wait for their loads
// at both ends of a tile (1000 tokens of 768 x 2048 both ways: 60 us of kernels, 315 TFLOP/s;
// float32, 1201 of 515 x 1365: 158 us, 64 TFLOP/s). A single token is bound by the weights'
// way from HBM: 4096 x 14336 44 us, 5.3 TB/s; up to 16 tokens 45, 64 tokens 51.
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

// s_waitcnt with vmcnt and lgkmcnt(0) (gfx9 encoding: vmcnt[3:0] bits 3:0, [5:4] bits 15:14)
#define MU_WAIT_VMCNT_LGKM0(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (((n) >> 4) << 14))

// A workgroup of four waves (two by two) for a tile, its slices through a ring of NS LDS
// slots that are loaded NS - 1 ahead, one barrier a slice. Slots are arrays of their own,
// so that the compiler's waits can tell a load into one from reads of another.
template <typename T, int MODE, int TS, int NS>
__global__ __launch_bounds__(NTHR, 1) void k_tile(TileArgs A) {
    constexpr bool DUAL = MODE == FWD || MODE == RECOMP;
    constexpr int ES = sizeof(T), BK = bk<T>(), WT = TS / 2, F = WT / 16, TN = DUAL ? TS / 2 : TS;
    typedef Operand<T, TS, MODE == DW> OA;
    typedef Operand<T, TS, MODE == DX || MODE == DW> OB;
    static_assert(NS == 2 || NS == 4, "ring of two or four");
    constexpr int SLOT = TS * 128, SPARE = NS == 4 ? SLOT : 16;
    __shared__ __attribute__((aligned(1024))) char sA0[SLOT];
    __shared__ __attribute__((aligned(1024))) char sA1[SLOT];
    __shared__ __attribute__((aligned(1024))) char sA2[SPARE];
    __shared__ __attribute__((aligned(1024))) char sA3[SPARE];
    __shared__ __attribute__((aligned(1024))) char sB0[SLOT];
    __shared__ __attribute__((aligned(1024))) char sB1[SLOT];
    __shared__ __attribute__((aligned(1024))) char sB2[SPARE];
    __shared__ __attribute__((aligned(1024))) char sB3[SPARE];
    auto slot_a = [&](auto st) -> char* {
        constexpr int S = decltype(st)::value;
        if constexpr (S == 0) return sA0;
        else if constexpr (S == 1) return sA1;
        else if constexpr (S == 2) return sA2;
        else return sA3;
    };
    auto slot_b = [&](auto st) -> char* {
        constexpr int S = decltype(st)::value;
        if constexpr (S == 0) return sB0;
        else if constexpr (S == 1) return sB1;
        else if constexpr (S == 2) return sB2;
        else return sB3;
    };

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

    // Where the tile's operands begin (DX: in dg and Wg, du and Wu; DUAL: in both weights),
    // the bytes of its rows (k along the rows) or what of a row lies before it (down the
    // rows), the bytes from slice to slice, and this lane's offsets in a slice. (A tile's
    // rows of at most 2^20 elements are within 2^30 bytes, so extents are 32 bits.)
    constexpr bool DOWN_A = MODE == DW, DOWN_B = MODE == DX || MODE == DW;
    const int64_t oa = DOWN_A ? m0 : m0 * A.lda, ob = DOWN_B ? n0 : n0 * A.ldb;
    const char* pa0 = (const char*)A.a[MODE == DW ? which : 0] + oa * ES;
    const char* pa1 = MODE == DX ? (const char*)A.a[1] + oa * ES : pa0;
    const char* pb0 = (const char*)A.b[0] + ob * ES;
    const char* pb1 = MODE == DX || DUAL ? (const char*)A.b[1] + ob * ES : pb0;
    const int a_bytes = DOWN_A ? (int)m0 * ES : (int)min(A.m - m0, (int64_t)TS) * (int)A.lda * ES;
    const int b_bytes = DOWN_B ? (int)n0 * ES : (int)min(A.n - n0, (int64_t)TN) * (int)A.ldb * ES;
    const int row_a = (int)A.lda * ES, row_b = (int)A.ldb * ES;
    int voA[OA::NI], voB[OB::NI];
#pragma unroll
    for (int i = 0; i < OA::NI; ++i) {
        const int r = OA::lds_row(i, wave, lane);
        voA[i] = r * row_a + OA::chunk(r, lane) * 16;
    }
#pragma unroll
    for (int i = 0; i < OB::NI; ++i) {
        const int r = OB::lds_row(i, wave, lane);
        // DUAL: LDS rows are, for each half of the columns, those of the gate and of the up projection
        voB[i] = (DUAL ? r / WT * (WT / 2) + r % (WT / 2) : r) * row_b + OB::chunk(r, lane) * 16;
    }
    const int chunk_k = (16 / ES) * ((lane & 7) ^ (lane >> 3));   // first k of this lane's chunk (k along the rows)
    // Direct loads of slice kt into a slot; behind the last slice nothing is read.
    auto dma = [&](auto st, int kt) {
        char *sa = slot_a(st), *sb = slot_b(st);
        const bool second = MODE == DX && kt >= kth;
        const int ks = second ? kt - kth : kt, left = (int)A.k - ks * BK;
        auto extent = [&](bool down, int row, int bytes) {
            return kt >= kt1 ? 0 : down ? min(left, BK) * row - bytes : bytes - ks * 128;
        };
        const int step_a = DOWN_A ? BK * row_a : 128, step_b = DOWN_B ? BK * row_b : 128;
        const int nb = extent(DOWN_B, row_b, b_bytes);
        __amdgpu_buffer_rsrc_t ra, rb, rb2;
        ra = resource((second ? pa1 : pa0) + (int64_t)ks * step_a, extent(DOWN_A, row_a, a_bytes));
        rb = resource((second ? pb1 : pb0) + (int64_t)ks * step_b, nb);
        rb2 = resource(pb1 + (int64_t)ks * step_b, nb);
#pragma unroll
        for (int i = 0; i < OA::NI; ++i) {
            const int off = DOWN_A || chunk_k < left ? voA[i] : OUTSIDE;
            char* dst = sa + (i * 4 + wave) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDSP void*)dst, 16, off, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < OB::NI; ++i) {
            const int off = DOWN_B || chunk_k < left ? voB[i] : OUTSIDE;
            char* dst = sb + (i * 4 + wave) * 1024;
            if (DUAL && (i * 32 + wave * 8) % WT / (WT / 2) == 1)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb2, (LDSP void*)dst, 16, off, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LDSP void*)dst, 16, off, 0, 0, 0);
        }
    };

    const int wm = (wave >> 1) * WT, wn = (wave & 1) * WT;
    f32x4 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // float32: a chain of instructions adds up 16 slices (512 k), the pieces are added up
    // behind each other. A sum of n independent terms is then off by at most 2^-24 sqrt((512 +
    // n / 512) / 6) of its size, in one chain by 2^-24 sqrt(n / 6): measured 0.41e-6 for 1.14e-6
    // at n = 4096. It costs the forward product of 4096 tokens, 2048 x 4096, 3 % (971 -> 1003
    // us; pieces of 256 4 %), most others 1 %. (Results of bfloat16 are rounded to 2^-8.)
    constexpr bool PIECES = ES == 4;
    f32x4 sums[PIECES ? F : 1][PIECES ? F : 1];
    if constexpr (PIECES) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) sums[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    int oa_r[4], ob_r[4];
    OA::offsets(oa_r, wm, lane);
    OB::offsets(ob_r, wn, lane);
    // (the weights' side first: a lane then holds four consecutive columns of a row)
    auto compute = [&](const char* sa, const char* sb) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            typename Mma<T>::Frag af[F], bf[F];
#pragma unroll
            for (int f = 0; f < F; ++f) bf[f] = OB::read(sb, ob_r, f, kk);
#pragma unroll
            for (int f = 0; f < F; ++f) af[f] = OA::read(sa, oa_r, f, kk);
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int j = 0; j < F; ++j) acc[i][j] = mma(bf[j], af[i], acc[i][j]);
        }
    };
    constexpr int LOADS = OA::NI + OB::NI;
    static_for<0, NS - 1>([&](auto s) { dma(s, kt0 + decltype(s)::value); });
    int kt = kt0;
    for (; kt + NS <= kt1; kt += NS) {
        static_for<0, NS>([&](auto s) {
            constexpr int S = decltype(s)::value;
            // this slice has landed and this wave's reads of the one before are done; a barrier
            // without __syncthreads' fence, which would wait for the loads on their way
            MU_WAIT_VMCNT_LGKM0((NS - 2) * LOADS);
            __builtin_amdgcn_s_barrier();
            dma(Stage<(S + NS - 1) % NS>{}, kt + S + NS - 1);
            compute(slot_a(s), slot_b(s));
        });
        if constexpr (PIECES) {
            if (((kt - kt0) & 15) == 16 - NS) {
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int j = 0; j < F; ++j) {
                        sums[i][j] += acc[i][j];
                        acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                    }
            }
        }
    }
    // the last few, all on their way
    MU_WAIT_VMCNT_LGKM0(0);
    __builtin_amdgcn_s_barrier();
    static_for<0, NS - 1>([&](auto s) {
        if (kt + decltype(s)::value < kt1) compute(slot_a(s), slot_b(s));
    });
    if constexpr (PIECES) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) acc[i][j] += sums[i][j];
    }

    // Results through LDS (a wave its own WT x WT block; the ring is done with), so that
    // they leave in runs of 8 columns of a row. Lane l holds columns 16 j + 4 (l >> 4) ..
    // +3 of row 16 i + (l & 15) of each fragment; 16-byte chunk c of row r lies at c ^ (r & 7).
    MU_WAIT_VMCNT_LGKM0(0);
    __syncthreads();
    float* st = (float*)(wave == 0 ? sA0 : wave == 1 ? sA1 : wave == 2 ? sB0 : sB1);
    static_assert(WT * WT * 4 <= SLOT, "a wave's block fits an array");
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
            *(f32x4*)(st + (i * 16 + (lane & 15)) * WT + (((j * 4 + (lane >> 4)) ^ (lane & 7)) << 2)) = acc[i][j];
    constexpr int CW = DUAL ? WT / 2 : WT, LPR = CW / 8, RPP = 64 / LPR;   // columns of a row, lanes of it, rows of a pass
    constexpr bool FAST = ES == 2;
    const int c = 2 * (lane % LPR);
    const int64_t col = n0 + (wave & 1) * CW + 4 * c;
    const int cnt = (int)min((int64_t)8, A.n - col);
#pragma clang loop unroll(disable)
    for (int p = 0; p < (WT + RPP - 1) / RPP; ++p) {
        const int r = p * RPP + lane / LPR;
        const int64_t row = m0 + wm + r;
        if (row >= A.m || cnt <= 0 || r >= WT) continue;
        const float* q = st + r * WT;
        auto run = [&](int chunk, float (&v)[8]) {
            const f32x4 x = *(const f32x4*)(q + ((chunk ^ (r & 7)) << 2)), y = *(const f32x4*)(q + (((chunk + 1) ^ (r & 7)) << 2));
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] = x[e]; v[e + 4] = y[e]; }
        };
        float v[8], w[8];
        run(c, v);
        if constexpr (DUAL) {
            run(CW / 4 + c, w);
            const int64_t at = row * A.ldo + col;
            float o[8], s[8];
            if constexpr (MODE == FWD) {
                if (A.gates[0]) {
                    if (ES == 2 && A.gates_f32) {
                        store_run<float, 8>((float*)A.gates[0] + at, cnt, v);
                        store_run<float, 8>((float*)A.gates[1] + at, cnt, w);
                    } else {
                        store_run<T, 8>((T*)A.gates[0] + at, cnt, v);
                        store_run<T, 8>((T*)A.gates[1] + at, cnt, w);
                    }
                }
                act_run<FAST>(A.act, v, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= w[e];
                store_run<T, 8>((T*)A.out[0] + at, cnt, o);
            } else {   // also the zeros behind rows that are padded to 16 bytes, which DX reads
                float d[8];
                load_run<T, 8>((const T*)A.dh + row * A.n + col, cnt, d);
                slope_run<FAST>(A.act, v, o, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[e] *= d[e] * w[e];
                    o[e] *= d[e];
                }
                const int put = (int)min((int64_t)8, A.ldo - col);
                store_run<T, 8>((T*)A.out[0] + at, put, s);
                store_run<T, 8>((T*)A.out[1] + at, put, o);
            }
        } else {
            const int64_t at = row * A.n + col;
            if (A.part) {
                const int64_t piece = MODE == DW ? blockIdx.y * 2 + which : blockIdx.y;
                store_run<float, 8>(A.part + piece * A.m * A.n + at, cnt, v);
            } else if (MODE == DW && (A.out_f32 || ES == 4)) {
                float* o = (float*)A.out[which] + at;
                if (A.accumulate) {
                    load_run<float, 8>(o, cnt, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += w[e];
                }
                store_run<float, 8>(o, cnt, v);
            } else {
                T* o = (T*)A.out[which] + at;
                if (MODE == DW && A.accumulate) {
                    load_run<T, 8>(o, cnt, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += w[e];
                }
                store_run<T, 8>(o, cnt, v);
            }
        }
    }
}

// Sums of the splits of a gradient, in order (of both weights', side by side in `part`);
// also zeros of both where there are no tokens.
struct JoinArgs {
    const float* part;
    void* out[2];
    int64_t n;        // elements of a result
    int splits;       // 0: zeros
    bool out_f32, accumulate;
};
__global__ __launch_bounds__(NTHR) void k_join(JoinArgs A) {
    const int64_t i = ((int64_t)blockIdx.x * NTHR + threadIdx.x) * 8;   // of one result (blockIdx.y)
    const int cnt = (int)min((int64_t)8, A.n - i);
    if (cnt <= 0) return;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8];
    for (int k = 0; k < A.splits; ++k) {
        load_run<float, 8>(A.part + ((int64_t)k * gridDim.y + blockIdx.y) * A.n + i, cnt, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
    void* out = blockIdx.y ? A.out[1] : A.out[0];
    if (A.accumulate) {
        if (A.out_f32) load_run<float, 8>((const float*)out + i, cnt, v);
        else load_run<bf16, 8>((const bf16*)out + i, cnt, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
    if (A.out_f32) store_run<float, 8>((float*)out + i, cnt, s);
    else store_run<bf16, 8>((bf16*)out + i, cnt, s);
}

// dg and du from the saved g and u, of type TG: rows of `n`, into rows of `pitch`, zeros behind.
// Columns lie along blockIdx.x and rows along blockIdx.y (a division for each run took as
// long as moving it; four rows a thread 238 us, one 204, for 8192 x 14336 bfloat16 with
// bfloat16 gates). HBM bound: five elements moved for each, 5.8 TB/s there; with float32
// gates 14 bytes for each, 312 us, 5.3 TB/s.
struct SlopeArgs {
    const void *dh, *g, *u;
    void *dg, *du;
    int64_t rows, n, pitch;
    int act;
};
template <typename T, typename TG>
__global__ __launch_bounds__(NTHR) void k_slopes(SlopeArgs A) {
    constexpr int V = vec_of<T>();
    const int64_t c = ((int64_t)blockIdx.x * NTHR + threadIdx.x) * V;
    const int cnt = (int)min((int64_t)V, A.n - c);
    if (c >= A.pitch) return;
    for (int64_t row = blockIdx.y; row < A.rows; row += gridDim.y) {
        const int64_t at = row * A.n + c;
        float d[V], g[V], u[V], a[V], s[V];
        load_run<T, V>((const T*)A.dh + at, cnt, d);
        load_run<TG, V>((const TG*)A.g + at, cnt, g);
        load_run<TG, V>((const TG*)A.u + at, cnt, u);
        slope_run<sizeof(T) == 2>(A.act, g, a, s);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s[e] = d[e] * u[e] * s[e];
            a[e] = d[e] * a[e];
        }
        store_run<T, V>((T*)A.dg + row * A.pitch + c, V, s);
        store_run<T, V>((T*)A.du + row * A.pitch + c, V, a);
    }
}

// Rows of n elements into rows of `pitch`, zeros behind them, of up to three matrices.
struct PackArgs {
    const void* src[3];
    void* dst[3];
    int64_t rows[3];
    int64_t n, pitch;
};
template <typename T>
__global__ __launch_bounds__(NTHR) void k_pack(PackArgs A) {
    constexpr int V = vec_of<T>();
    const int64_t c = ((int64_t)blockIdx.x * NTHR + threadIdx.x) * V;
    if (c >= A.pitch) return;
    const int m = blockIdx.z;
    const T* src = (const T*)(m == 0 ? A.src[0] : m == 1 ? A.src[1] : A.src[2]);
    T* dst = (T*)(m == 0 ? A.dst[0] : m == 1 ? A.dst[1] : A.dst[2]);
    const int64_t rows = m == 0 ? A.rows[0] : m == 1 ? A.rows[1] : A.rows[2];
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        float v[V];
        load_run<T, V>(src + row * A.n + c, (int)min((int64_t)V, A.n - c), v);
        store_run<T, V>(dst + row * A.pitch + c, V, v);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
size_t es_of(int dtype) { return dtype == MU_BF16 ? 2 : 4; }
bool gates_f32(int dtype, int activation) { return dtype == MU_F32 || (activation & MU_GATES_F32); }
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An operand: where it lies, or the place of its padded copy in the workspace.
struct Source {
    const void* p;
    int64_t rows, n, pitch;
    bool copied;
    size_t off;
};

// How a product is cut: the tile's edge, and the slices of k of a workgroup.
struct Cut {
    int edge, kt, splits;
};

struct Plan {
    Source x, wg, wu;
    size_t off_dg, off_du, off_part, bytes;
    int64_t pitch_h;                    // of dg and du
    Cut fwd, dx, dw;
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

int64_t tiles_of(int64_t m, int64_t n, int nmat, bool dual, int edge) {
    return nmat * ceil_div(m, edge) * ceil_div(n, dual ? edge / 2 : edge);
}

// Tiles of 256 (bfloat16) where they fill half the chip. There they are level with those of
// 128: forward of 1024 tokens of 4096 x 4096 (128 tiles) 81 us, 78 with 128; gradient of x of
// 2048 of 4096 x 14336 (128) 490, 503. In whole rounds of 256 tiles they run at 1.5 times the
// rate (forward of 8192 of 4096 x 14336 1417, 2083) and in between mostly ahead (352 tiles, the
// weights' gradients of 2048 x 5632, 100, 120; 288, forward of 2300 of 4096 x 4096, 177, 177),
// but not just past a round (266 tiles, the weights' gradients of 1600 x 4800, 235, 200). Else
// 128 where those give every compute unit one, and 64. Measured on
// kernels of 768 x 2048 (bfloat16, us, edge 64 against 128): forward of 1000 tokens
// 15.4, 13.8 (256 tiles of 128), of 256 tokens 6.3, 11.1 (64); both weights' gradients
// 15, 17 (192) and 4.4, 4.8 (192); 64 tokens of 4096 x 14336 131, 121 (7168).
//
// The gradient of x is split over k (2 * hidden): its tiles are few and their k long. The
// weights' gradients are large and few k deep (splitting those in two cost 1000 tokens 10
// us, 512 tokens of 2048 x 8192 105), unless their tiles leave half the chip idle: 16384
// tokens of 256 x 512 (64 tiles of 64) 72 against 46 us, float32 299 against 108; 1024
// tokens 11.3 against 12.5, so bfloat16 splits have sixteen slices at least. As many splits as fill the chip twice (two
// workgroups of 64 a compute unit), else eight slices at least: 256 tokens of 768 x 2048,
// 48 tiles, 1, 2, 4 splits 21.9, 18.1, 16.6 us, float32 78, 47, 31; 64 tokens of 4096 x
// 14336, 64 tiles, 103, 60, 38.5; 1000 tokens of 768, float32, 192 tiles, 82, 78, 66.
Cut cut_of(int64_t m, int64_t n, int nmat, bool dual, int64_t kts, int dtype, bool split) {
    auto tiles = [&](int e) { return tiles_of(m, n, nmat, dual, e); };
    Cut c{128, (int)kts, 1};
    if (dtype == MU_BF16 && tiles(256) >= 128) c.edge = 256;
    else if (tiles(128) < 256) c.edge = 64;
    if (split && nmat == 1 && dtype == MU_BF16 && c.edge == 64 && tiles(128) >= 96 && kts >= 32) {
        c.edge = 128;   // 2048 tokens of 1000 x 2500: two splits of 128 51 us, tiles of 64 60
        c.splits = 2;
    } else if (split && c.edge == 64 && tiles(64) < (nmat == 2 ? 128 : 384)) {
        c.splits = (int)std::max<int64_t>(1, std::min<int64_t>({ceil_div(512, tiles(64)), kts / (nmat == 2 && dtype == MU_BF16 ? 16 : 8), 16}));
    }
    c.kt = (int)ceil_div(kts, c.splits);
    c.splits = (int)ceil_div(kts, c.kt);
    return c;
}

Plan plan_fwd(const mu_gated* a) {
    Plan p{};
    const int es = (int)es_of(a->dtype);
    p.x = source(a->x, a->tokens, a->dim, es, p);
    p.wg = source(a->w_gate, a->hidden, a->dim, es, p);
    p.wu = source(a->w_up, a->hidden, a->dim, es, p);
    p.fwd = cut_of(a->tokens, a->hidden, 1, true, ceil_div(a->dim, 128 / es), a->dtype, false);
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
    p.fwd = cut_of(a->tokens, a->hidden, 1, true, ceil_div(a->dim, bk), a->dtype, false);
    p.dx = cut_of(a->tokens, a->dim, 1, false, 2 * ceil_div(a->hidden, bk), a->dtype, true);
    p.dw = cut_of(a->hidden, a->dim, 2, false, ceil_div(a->tokens, bk), a->dtype, true);
    size_t part = 0;
    if (a->dx && p.dx.splits > 1) part = sizeof(float) * (size_t)(p.dx.splits * a->tokens * a->dim);
    if (a->d_gate && p.dw.splits > 1) part = std::max(part, sizeof(float) * (size_t)(p.dw.splits * 2 * a->hidden * a->dim));
    p.off_part = p.bytes;
    p.bytes += align_up(part);
    return p;
}

// What a call launches fits its grids: seen before the first of its launches.
constexpr int64_t MAX_TILES = 1 << 23, MAX_JOIN_WGS = (1 << 24) - 1;
int check_plan(const mu_gated* a, const Plan& p) {
    if (tiles_of(a->tokens, a->hidden, 1, true, p.fwd.edge) > MAX_TILES) return fail(MU_ERR_INVALID_ARG, "too many tiles for one launch");
    return MU_OK;
}
int check_plan(const mu_gated_grad* a, const Plan& p) {
    if ((!a->gate && tiles_of(a->tokens, a->hidden, 1, true, p.fwd.edge) > MAX_TILES) ||
        (a->dx && tiles_of(a->tokens, a->dim, 1, false, p.dx.edge) > MAX_TILES) ||
        (a->d_gate && tiles_of(a->hidden, a->dim, 2, false, p.dw.edge) > MAX_TILES))
        return fail(MU_ERR_INVALID_ARG, "too many tiles for one launch");
    return MU_OK;
}

const void* at(const Source& s, const char* ws) { return s.copied ? ws + s.off : s.p; }

// The padded copies of a call, one launch.
template <typename T>
int pack(int kernel, const Plan& p, char* ws, hipStream_t st) {
    PackArgs a{};
    int n = 0;
    int64_t rows = 0;
    for (const Source* s : {&p.x, &p.wg, &p.wu}) {
        if (!s->copied) continue;
        a.src[n] = s->p;
        a.dst[n] = ws + s->off;
        a.rows[n++] = s->rows;
        a.n = s->n;
        a.pitch = s->pitch;
        rows = std::max(rows, s->rows);
    }
    if (n == 0) return MU_OK;
    return timed_launch(kernel, 0.0, 0.0, st, [&] {
        const dim3 grid((unsigned)ceil_div(a.pitch, vec_of<T>() * NTHR), (unsigned)std::min<int64_t>(rows, 4096), (unsigned)n);
        hipLaunchKernelGGL(k_pack<T>, grid, dim3(NTHR), 0, st, a);
        return hipGetLastError();
    }, "operand copy launch");
}

template <typename T, int MODE>
int product(int kernel, TileArgs a, const Cut& c, double flops, double bytes, hipStream_t s) {
    const int64_t tm = ceil_div(a.m, c.edge) * (MODE == DW ? 2 : 1);
    const int64_t tn = ceil_div(a.n, MODE == FWD || MODE == RECOMP ? c.edge / 2 : c.edge);
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    a.kt_split = c.kt;
    a.aligned = a.n % 8 == 0 && a.ldo % 8 == 0;
    for (const void* p : {(const void*)a.out[0], (const void*)a.out[1], (const void*)a.gates[0], (const void*)a.gates[1]})
        a.aligned = a.aligned && aligned(p, 16);
    return timed_launch(kernel, flops, bytes, s, [&] {
        if (c.edge == 256) return launch_wide(MODE, a, (int)std::min<int64_t>(256, round_up(tm * tn, 8)), s);
        const dim3 grid((unsigned)round_up(tm * tn, 8), (unsigned)c.splits);
        if (c.edge == 128) hipLaunchKernelGGL((k_tile<T, MODE, 128, sizeof(T) == 2 ? 4 : 2>), grid, dim3(NTHR), 0, s, a);
        else hipLaunchKernelGGL((k_tile<T, MODE, 64, 4>), grid, dim3(NTHR), 0, s, a);
        return hipGetLastError();
    }, "gated feed-forward product launch");
}

int join(const JoinArgs& j, hipStream_t s) {
    const int64_t wgs = ceil_div(j.n, 8 * NTHR);   // (within MAX_JOIN_WGS: splits have few tiles, zeros are checked)
    return timed_launch(MU_K_GATED_GRAD, 0.0, 0.0, s, [&] {
        hipLaunchKernelGGL(k_join, dim3((unsigned)wgs, j.out[1] ? 2 : 1), dim3(NTHR), 0, s, j);
        return hipGetLastError();
    }, "gated feed-forward join launch");
}

template <typename T>
int run_fwd(const mu_gated* a, const Plan& p, char* ws, hipStream_t s) {
    const int rc = pack<T>(MU_K_GATED, p, ws, s);
    if (rc) return rc;
    TileArgs t{};
    t.a[0] = at(p.x, ws);
    t.b[0] = at(p.wg, ws);
    t.b[1] = at(p.wu, ws);
    t.lda = p.x.pitch;
    t.ldb = p.wg.pitch;
    t.m = a->tokens;
    t.n = a->hidden;
    t.k = a->dim;
    t.act = a->activation & ~MU_GATES_F32;
    t.out[0] = a->h;
    t.ldo = a->hidden;
    t.gates[0] = a->gate_out;
    t.gates[1] = a->up_out;
    t.gates_f32 = gates_f32(a->dtype, a->activation);
    const double n = (double)a->tokens, d = (double)a->dim, f = (double)a->hidden;
    return product<T, FWD>(MU_K_GATED, t, p.fwd, 4.0 * n * d * f,
                           sizeof(T) * (n * d + 2 * d * f + n * f) + (a->gate_out ? (t.gates_f32 ? 8 : 4) * n * f : 0.0), s);
}

template <typename T>
int run_bwd(const mu_gated_grad* a, const Plan& p, char* ws, hipStream_t s) {
    const double n = (double)a->tokens, d = (double)a->dim, f = (double)a->hidden;
    int rc = pack<T>(MU_K_GATED_GRAD, p, ws, s);
    if (rc) return rc;
    T *dg = (T*)(ws + p.off_dg), *du = (T*)(ws + p.off_du);
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
        t.act = a->activation & ~MU_GATES_F32;
        t.dh = a->grad_h;
        t.out[0] = dg;
        t.out[1] = du;
        t.ldo = p.pitch_h;
        rc = product<T, RECOMP>(MU_K_GATED_GRAD, t, p.fwd, 4.0 * n * d * f, sizeof(T) * (n * d + 2 * d * f + 3 * n * f), s);
    } else {
        const bool f32 = gates_f32(a->dtype, a->activation);
        rc = timed_launch(MU_K_GATED_GRAD, 0.0, (3.0 * sizeof(T) + (f32 ? 8 : 4)) * n * f, s, [&] {
            const dim3 grid((unsigned)ceil_div(p.pitch_h, vec_of<T>() * NTHR),
                            (unsigned)std::min<int64_t>(a->tokens, 65535));
            const SlopeArgs sa{a->grad_h, a->gate, a->up, dg, du, a->tokens, a->hidden, p.pitch_h, a->activation & ~MU_GATES_F32};
            if (f32) hipLaunchKernelGGL((k_slopes<T, float>), grid, dim3(NTHR), 0, s, sa);
            else hipLaunchKernelGGL((k_slopes<T, T>), grid, dim3(NTHR), 0, s, sa);
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
        t.out[0] = a->dx;
        t.part = p.dx.splits > 1 ? (float*)(ws + p.off_part) : nullptr;
        rc = product<T, DX>(MU_K_GATED_GRAD, t, p.dx, 4.0 * n * d * f, sizeof(T) * (n * d + 2 * d * f + 2 * n * f), s);
        if (!rc && t.part) rc = join(JoinArgs{t.part, {a->dx, nullptr}, a->tokens * a->dim, p.dx.splits, sizeof(T) == 4, false}, s);
        if (rc) return rc;
    }
    if (a->d_gate) {
        t.b[0] = at(p.x, ws);
        t.ldb = p.x.pitch;
        t.m = a->hidden;
        t.n = a->dim;
        t.k = a->tokens;
        t.out[0] = a->d_gate;
        t.out[1] = a->d_up;
        t.out_f32 = a->grad_dtype == MU_F32;
        t.accumulate = a->accumulate;
        t.part = p.dw.splits > 1 ? (float*)(ws + p.off_part) : nullptr;
        rc = product<T, DW>(MU_K_GATED_GRAD, t, p.dw, 4.0 * n * d * f,
                            sizeof(T) * (n * d + 2 * n * f) + es_of(a->grad_dtype) * 2 * d * f, s);
        if (!rc && t.part)
            rc = join(JoinArgs{t.part, {a->d_gate, a->d_up}, a->hidden * a->dim, p.dw.splits, t.out_f32, t.accumulate != 0}, s);
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
    const int kind = act & ~MU_GATES_F32;
    if (kind < MU_ACT_SILU || kind > MU_ACT_RELU) return fail(MU_ERR_INVALID_ARG, "unknown activation %d", act);
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
    const size_t es = es_of(a->dtype), ega = gates_f32(a->dtype, a->activation) ? 4 : 2;
    const int64_t nx = a->tokens * a->dim, nw = a->hidden * a->dim, nh = a->tokens * a->hidden;
    return check_buffers({Buf{a->x, nx, es}, Buf{a->w_gate, nw, es}, Buf{a->w_up, nw, es}},
                         {Buf{a->h, nh, es}, Buf{a->gate_out, nh, ega}, Buf{a->up_out, nh, ega}});
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
    if (a->tokens == 0 && a->d_gate && !a->accumulate && ceil_div(a->hidden * a->dim, 8 * NTHR) > MAX_JOIN_WGS)
        return fail(MU_ERR_INVALID_ARG, "too many elements for one launch");
    const size_t es = es_of(a->dtype), eg = es_of(a->grad_dtype), ega = gates_f32(a->dtype, a->activation) ? 4 : 2;
    const int64_t nx = a->tokens * a->dim, nw = a->hidden * a->dim, nh = a->tokens * a->hidden;
    return check_buffers({Buf{a->grad_h, nh, es}, Buf{a->x, nx, es}, Buf{a->w_gate, nw, es}, Buf{a->w_up, nw, es},
                          Buf{a->gate, nh, ega}, Buf{a->up, nh, ega}},
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
        const Plan p = a->tokens == 0 ? Plan{} : plan_fwd(a);
        *bytes = p.bytes;
        return a->tokens == 0 ? MU_OK : check_plan(a, p);
    });
}

int mu_gated_mlp(const mu_gated* a, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_fwd(a);
        if (rc || a->tokens == 0) return rc;
        const Plan p = plan_fwd(a);
        rc = check_plan(a, p);
        if (!rc) rc = check_workspace(ws, ws_bytes, p.bytes);
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
        const Plan p = a->tokens == 0 ? Plan{} : plan_bwd(a);
        *bytes = p.bytes;
        return a->tokens == 0 ? MU_OK : check_plan(a, p);
    });
}

int mu_gated_mlp_grad(const mu_gated_grad* a, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_bwd(a);
        if (rc || (!a->dx && !a->d_gate)) return rc;
        hipStream_t s = (hipStream_t)stream;
        if (a->tokens == 0) {   // no rows: zero gradients
            if (!a->d_gate || a->accumulate) return MU_OK;
            return join(JoinArgs{nullptr, {a->d_gate, a->d_up}, a->hidden * a->dim, 0, a->grad_dtype == MU_F32, false}, s);
        }
        const Plan p = plan_bwd(a);
        rc = check_plan(a, p);
        if (!rc) rc = check_workspace(ws, ws_bytes, p.bytes);
        if (rc) return rc;
        return a->dtype == MU_BF16 ? run_bwd<bf16>(a, p, (char*)ws, s) : run_bwd<float>(a, p, (char*)ws, s);
    });
}

}  // extern "C"
