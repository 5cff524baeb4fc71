// The gated feed-forward block's products in tiles of 256 x 256 (bfloat16).
//
// Four waves of 128 x 128, each with its 256 accumulators pinned in the second
// register file. A slice of 64 k of both operands is 64 KB of LDS, and there are two
// such slots; rows of 64 k are 128 bytes, whole lines. (Slices of 32 k with four
// slots, as the square products of the Newton-Schulz steps have them, would fetch
// every line of operands in their own layouts twice.)
//
// A wave multiplies a slice in four phases of 32 matrix instructions, by halves A0,
// A1 of its rows and B0, B1 of its columns: A0 B0, A0 B1, A1 B1, A1 B0. In each phase
// one half is new and one is dead, so each phase reads the half that the next one
// needs into the registers of the dead one, four halves of 32 registers in all:
//   phase 0   A0 B0   reads B1               loads A0 of the slice after next
//   phase 1   A0 B1   reads A1               loads B0
//   phase 2   A1 B1   reads A0 of the next   loads B1
//   phase 3   A1 B0   reads B0 of the next   loads A1
// A half's place in LDS is loaded again as soon as it has been read, so a load has
// five phases and more (2500 cycles) to arrive. Two barriers a slice, in phases 1
// and 3 behind their first eight instructions: what was read before one may be
// overwritten behind it, and what the next two phases read has landed (the 16
// youngest loads may still be on their way). Reads, loads and instructions are
// spread evenly, in a fixed order: as one wave a SIMD leaves nothing else to run, a
// burst of either stalls the wave (all 16 loads of a slice in 48 instructions: 1.03
// to 1.15 PFLOP/s).
//
// A workgroup takes tile after tile (one fixed share each, those of an XCD next to
// each other) and starts the loads of the next tile before it writes this one.
//
// What bounds it: matrix instructions, 2048 cycles of a slice. With its share of the results
// a slice of the gradients takes 2620 to 2650 (896 slices and 2 or 7 tiles a workgroup); of
// the forward product with float32 gates, 14 tiles, 3140, without gates 2870. 8192 tokens of
// 4096 x 14336: gradient of x 1340 to 1390 us, of both weights 1360 to 1430 (1.35 to 1.43
// PFLOP/s at 1.7 GHz, the clock under this load), forward 1385 to 1415 without gates, 1520 to
// 1650 with float32 ones. Both ways with bfloat16 gates in tiles of 128 with two barriers a
// slice 6550, with these 4390.
#include "gated.hpp"

namespace mu {
namespace gated {

namespace {

// s_waitcnt with vmcnt(0) and lgkmcnt(0)
#define MU_WAIT_ALL() __builtin_amdgcn_s_waitcnt((7 << 4))

// Four accumulators of a lane to LDS, straight from their registers. (The strip is named
// so that the compiler does not make one write of eight, which would copy the
// accumulators to common registers first.)
template <int STRIP, int OFF>
__device__ __forceinline__ void put_acc(const f32x4& c, uint32_t at) {
    asm volatile("ds_write_b128 %1, %0 offset:%c2 ; strip %c3" : : "a"(c), "v"(at), "n"(OFF), "n"(STRIP) : "memory");
}

// Half p of an operand's slice in LDS: for each wave half w (rows or columns 128 w ..)
// 64 rows of 128 bytes, rows of the operand with 64 k, or (DOWN) k with 64 columns.
// 16-byte chunks are permuted so that reads touch all banks.
template <bool DOWN>
struct Half {
    // chunk of the operand's row (of 8 in 128 bytes) that lies at place `at` of LDS row r
    __device__ static __forceinline__ int chunk(int r, int at) {
        return DOWN ? at ^ (((r >> 1) & 1) << 1 | ((r >> 3) & 1) << 2) : at ^ (r & 7);
    }
    // This lane's offsets in the reads of a half: from `at` bytes on, for each k half of rows,
    // or for each 16 columns (DOWN). Opaque, so that each address is an array, one of these
    // and a constant: the compiler's alias analysis follows an address over a few steps
    // only, and where it loses it a read waits for every load on its way.
    __device__ static __forceinline__ void offsets(int (&o)[4], int at, int lane) {
        const int i = lane & 15, g = lane >> 4;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if constexpr (DOWN) {
                // lane i of 16 addresses 4 columns of k row i / 4 and receives column i of
                // those four rows (ds_read_b64_tr_b16)
                const int r = 8 * g + (i >> 2);
                o[n] = at + r * 128 + (chunk(r, 2 * n) + ((i >> 1) & 1)) * 16 + 8 * (i & 1);
            } else {
                o[n] = at + i * 128 + ((((n & 1) * 4 + g) ^ (i & 7)) << 4);
            }
            asm("" : "+v"(o[n]));
        }
    }
    // Fragment f (16 rows or columns) of k half kk.
    __device__ static __forceinline__ bf16x8 read(const char* lds, const int (&o)[4], int f, int kk) {
        if constexpr (!DOWN) {
            return *(const bf16x8*)(lds + o[kk] + f * 2048);
        } else {
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDSP i16x4*)(lds + o[f] + kk * 4096));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDSP i16x4*)(lds + o[f] + (kk * 4096 + 512)));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

template <int MODE>
__global__ __launch_bounds__(NTHR, 1) void k_wide(TileArgs A) {
    constexpr bool DUAL = MODE == FWD || MODE == RECOMP;
    constexpr bool DOWN_A = MODE == DW, DOWN_B = MODE == DX || MODE == DW;
    constexpr int TS = 256, WT = 128, F = 8, H = F / 2, TN = DUAL ? 128 : 256;
    typedef Half<DOWN_A> HA;
    typedef Half<DOWN_B> HB;
    // slot and half; arrays of their own, so that the compiler's waits can tell a load
    // into one from reads of another
    __shared__ __attribute__((aligned(1024))) char sA00[16384];
    __shared__ __attribute__((aligned(1024))) char sA01[16384];
    __shared__ __attribute__((aligned(1024))) char sA10[16384];
    __shared__ __attribute__((aligned(1024))) char sA11[16384];
    __shared__ __attribute__((aligned(1024))) char sB00[16384];
    __shared__ __attribute__((aligned(1024))) char sB01[16384];
    __shared__ __attribute__((aligned(1024))) char sB10[16384];
    __shared__ __attribute__((aligned(1024))) char sB11[16384];
    __shared__ __attribute__((aligned(1024))) float sE[4][16 * 128];   // a strip of 16 rows for each wave's results

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave >> 1) * WT, wn = (wave & 1) * WT;
    const int total = A.tiles_m * A.tiles_n;
    const int kth = (int)((A.k + 63) / 64), KT = MODE == DX ? 2 * kth : kth;

    // This lane's offsets within a slice: load j of half p fills 1 KB, eight LDS rows
    // from 8 (4 (j & 1) + wave) on of wave half j / 2.
    int voA[2][4], voB[2][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * (4 * (j & 1) + wave) + (lane >> 3), w = j >> 1;
            const int ca = HA::chunk(r, lane & 7), cb = HB::chunk(r, lane & 7);
            voA[p][j] = DOWN_A ? r * (int)A.lda * 2 + (w * 128 + p * 64) * 2 + ca * 16 : (w * 128 + p * 64 + r) * (int)A.lda * 2 + ca * 16;
            // DUAL: half 0 of the columns are the gate's, half 1 the up projection's
            voB[p][j] = DOWN_B ? r * (int)A.ldb * 2 + (w * 128 + p * 64) * 2 + cb * 16
                      : DUAL   ? (w * 64 + r) * (int)A.ldb * 2 + cb * 16
                               : (w * 128 + p * 64 + r) * (int)A.ldb * 2 + cb * 16;
        }
    int oa[4], ob[4];
    HA::offsets(oa, (wave >> 1) * 8192, lane);
    HB::offsets(ob, (wave & 1) * 8192, lane);
    const int chunk_k = 8 * ((lane & 7) ^ (lane >> 3));   // first k of this lane's chunk (k along the rows)

    // Tiles: XCD x takes a contiguous share, its workgroups the next of it in turn.
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, per_xcd = gridDim.x >> 3;
    const int share = (total + 7) / 8, t_end = min(total, (xcd + 1) * share);

    // The tile: its place, where its operands begin (DX: in dg and Wg, du and Wu; DUAL:
    // in the gate's and the up projection's weights), and the bytes of its rows (k along
    // the rows) or what of a row lies before it (DOWN).
    int which = 0, a_bytes = 0, b_bytes = 0;
    int64_t m0 = 0, n0 = 0;
    const char *pa0 = nullptr, *pa1 = nullptr, *pb0 = nullptr, *pb1 = nullptr;
    auto place = [&](int t) {
        int ti, tj;
        tile_of(t, A.tiles_m, A.tiles_n, ti, tj);
        which = 0;
        if (MODE == DW && ti >= A.tiles_m / 2) {
            which = 1;
            ti -= A.tiles_m / 2;
        }
        m0 = (int64_t)ti * TS;
        n0 = (int64_t)tj * TN;
        const int64_t oa = DOWN_A ? m0 : m0 * A.lda, ob = DOWN_B ? n0 : n0 * A.ldb;
        pa0 = (const char*)A.a[MODE == DW ? which : 0] + oa * 2;
        pa1 = MODE == DX ? (const char*)A.a[1] + oa * 2 : pa0;
        pb0 = (const char*)A.b[0] + ob * 2;
        pb1 = MODE == DX || DUAL ? (const char*)A.b[1] + ob * 2 : pb0;
        a_bytes = DOWN_A ? (int)m0 * 2 : (int)min(A.m - m0, (int64_t)TS) * (int)A.lda * 2;
        b_bytes = DOWN_B ? (int)n0 * 2 : (int)min(A.n - n0, (int64_t)TN) * (int)A.ldb * 2;
    };
    const int step_a = DOWN_A ? 128 * (int)A.lda : 128, step_b = DOWN_B ? 128 * (int)A.ldb : 128;   // bytes of a slice

    auto at_a = [&](auto st, auto pc) -> char* {
        constexpr int n = decltype(st)::value * 2 + decltype(pc)::value;
        if constexpr (n == 0) return sA00;
        else if constexpr (n == 1) return sA01;
        else if constexpr (n == 2) return sA10;
        else return sA11;
    };
    auto at_b = [&](auto st, auto pc) -> char* {
        constexpr int n = decltype(st)::value * 2 + decltype(pc)::value;
        if constexpr (n == 0) return sB00;
        else if constexpr (n == 1) return sB01;
        else if constexpr (n == 2) return sB10;
        else return sB11;
    };

    // fn(resource, k that are left) of slice kt of one operand (B: its half p); beyond the
    // last slice nothing is read. (A tile's rows of at most 2^20 elements are within 2^29
    // bytes, so extents are 32 bits.)
    auto with = [&](bool down, int kt, const char* p0, const char* p1, int step, int bytes, auto&& fn) {
        const bool second = MODE == DX && kt >= kth;
        const int ks = second ? kt - kth : kt, left = (int)A.k - ks * 64;
        const int n = down ? min(left, 64) * (step >> 6) - bytes : bytes - ks * 128;
        fn(resource((second ? p1 : p0) + (int64_t)ks * step, kt < KT ? n : 0), left);
    };
    auto with_a = [&](int kt, auto&& fn) { with(DOWN_A, kt, pa0, pa1, step_a, a_bytes, fn); };
    auto with_b = [&](int kt, auto pc, auto&& fn) {
        if constexpr (DUAL && decltype(pc)::value == 1) with(DOWN_B, kt, pb1, pb1, step_b, b_bytes, fn);
        else with(DOWN_B, kt, pb0, pb1, step_b, b_bytes, fn);
    };
    // (where a load goes is added up at each one: held ready for all, 32 places and what
    // they crowd out cost lane reads in the loop)
    auto load_a = [&](auto st, auto pc, auto jc, __amdgpu_buffer_rsrc_t rs, int left) {
        constexpr int p = decltype(pc)::value, j = decltype(jc)::value;
        const int off = DOWN_A || chunk_k < left ? voA[p][j] : OUTSIDE;
        int w = wave * 1024;
        asm volatile("" : "+s"(w));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDSP void*)(at_a(st, pc) + w + ((j >> 1) * 8192 + (j & 1) * 4096)), 16, off, 0, 0, 0);
    };
    auto load_b = [&](auto st, auto pc, auto jc, __amdgpu_buffer_rsrc_t rs, int left) {
        constexpr int p = decltype(pc)::value, j = decltype(jc)::value;
        const int off = DOWN_B || chunk_k < left ? voB[p][j] : OUTSIDE;
        int w = wave * 1024;
        asm volatile("" : "+s"(w));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDSP void*)(at_b(st, pc) + w + ((j >> 1) * 8192 + (j & 1) * 4096)), 16, off, 0, 0, 0);
    };
    auto half_a = [&](auto st, auto pc, int kt) {
        with_a(kt, [&](auto rs, int left) { static_for<0, 4>([&](auto j) { load_a(st, pc, j, rs, left); }); });
    };
    auto half_b = [&](auto st, auto pc, int kt) {
        with_b(kt, pc, [&](auto rs, int left) { static_for<0, 4>([&](auto j) { load_b(st, pc, j, rs, left); }); });
    };

    f32x4 acc[F][F];
    bf16x8 P[2 * H], Q[2 * H], X[2 * H], Y[2 * H];   // halves: fragment f of k half kk at 4 kk + f

    // Matrix instruction n of a phase (k half by k half, row by row of the fragments) on
    // the halves pa, pb. Written out, so that the accumulators stay where they are.
    auto mul_acc = [](auto nc, auto pac, auto pbc, f32x4 (&c)[F][F], const bf16x8 (&a)[2 * H], const bf16x8 (&b)[2 * H]) {
        constexpr int n = decltype(nc)::value, kk = n / 16, i = n / 4 % 4, j = n % 4;
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0"
                     : "+a"(c[decltype(pac)::value * 4 + i][decltype(pbc)::value * 4 + j])
                     : "v"(b[4 * kk + j]), "v"(a[4 * kk + i]));
    };
    // One phase: the products of a and b; read(g) reads fragment g of eight, load(j) is
    // load j of four. SYNC: the barrier behind the first eight products.
    auto phase = [&](auto sync, auto pac, auto pbc, const bf16x8 (&a)[2 * H], const bf16x8 (&b)[2 * H], auto&& read, auto&& load) {
        constexpr int HEAD = decltype(sync)::value ? 8 : 0;
        auto mul = [&](auto n) { mul_acc(n, pac, pbc, acc, a, b); };
        if constexpr (HEAD > 0) {
            static_for<0, HEAD>(mul);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt((16 & 15) | (7 << 4) | ((16 >> 4) << 14));   // vmcnt(16), lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
        }
        static_for<0, 8>([&](auto gc) {
            constexpr int g = decltype(gc)::value, per = (32 - HEAD) / 8;
            read(gc);
            if constexpr (g % 2 == 0) load(Stage<g / 2>{});
            static_for<HEAD + g * per, HEAD + (g + 1) * per>(mul);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // Slice kt in slot S; B0 is in X and B1 goes to Y, or (SWAP) the other way round.
    auto slice = [&](auto st, int kt, bf16x8 (&b0)[2 * H], bf16x8 (&b1)[2 * H]) {
        constexpr int S = decltype(st)::value;
        using SN = Stage<1 - S>;
        typedef Stage<0> C0;
        typedef Stage<1> C1;
        with_a(kt + 2, [&](auto rs, int left) {
            phase(C0{}, C0{}, C0{}, P, b0, [&](auto g) { b1[g.value] = HB::read(at_b(st, C1{}), ob, g.value % 4, g.value / 4); },
                  [&](auto j) { load_a(st, C0{}, j, rs, left); });
        });
        with_b(kt + 2, C0{}, [&](auto rs, int left) {
            phase(C1{}, C0{}, C1{}, P, b1, [&](auto g) { Q[g.value] = HA::read(at_a(st, C1{}), oa, g.value % 4, g.value / 4); },
                  [&](auto j) { load_b(st, C0{}, j, rs, left); });
        });
        with_b(kt + 2, C1{}, [&](auto rs, int left) {
            phase(C0{}, C1{}, C1{}, Q, b1, [&](auto g) { P[g.value] = HA::read(at_a(SN{}, C0{}), oa, g.value % 4, g.value / 4); },
                  [&](auto j) { load_b(st, C1{}, j, rs, left); });
        });
        with_a(kt + 2, [&](auto rs, int left) {
            phase(C1{}, C1{}, C0{}, Q, b0, [&](auto g) { b1[g.value] = HB::read(at_b(SN{}, C0{}), ob, g.value % 4, g.value / 4); },
                  [&](auto j) { load_a(st, C1{}, j, rs, left); });
        });
    };
    // The loads of a tile that its first phases do not make themselves, by eighths.
    auto start = [&](auto nc) {
        constexpr int n = decltype(nc)::value;
        typedef Stage<0> C0;
        typedef Stage<1> C1;
        if constexpr (n == 0) half_a(C0{}, C0{}, 0);
        else if constexpr (n == 1) half_b(C0{}, C0{}, 0);
        else if constexpr (n == 2) half_b(C0{}, C1{}, 0);
        else if constexpr (n == 3) half_a(C0{}, C1{}, 0);
        else if constexpr (n == 4) half_a(C1{}, C0{}, 1);
        else if constexpr (n == 5) half_b(C1{}, C0{}, 1);
        else if constexpr (n == 6) half_b(C1{}, C1{}, 1);
        else half_a(C1{}, C1{}, 1);
    };

    int t = xcd * share + slot;
    if (t >= t_end) return;
    place(t);
    static_for<0, 8>(start);
    for (;;) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        // A0, B0 and B1 of the first slice; 20 loads may still be on their way
        __builtin_amdgcn_s_waitcnt((20 & 15) | (7 << 4) | (15 << 8) | ((20 >> 4) << 14));
        __builtin_amdgcn_s_barrier();
        static_for<0, 8>([&](auto g) {
            constexpr int G = decltype(g)::value;
            P[G] = HA::read(sA00, oa, G % 4, G / 4);
            X[G] = HB::read(sB00, ob, G % 4, G / 4);
        });
        __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));   // lgkmcnt(0): A0's place is loaded again in the first phase
        __builtin_amdgcn_s_barrier();
        asm volatile("s_nop 1");   // accumulators just written, which the compiler cannot see
        __builtin_amdgcn_sched_barrier(0);
        for (int kt = 0; kt < KT; kt += 2) {
            slice(Stage<0>{}, kt, X, Y);
            slice(Stage<1>{}, kt + 1, Y, X);
        }
        // the last matrix instructions' wait states, which the compiler cannot see
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        MU_WAIT_ALL();
        __builtin_amdgcn_s_barrier();   // nobody reads the slots any more

        const int64_t row0 = m0 + wm, col0 = n0 + (DUAL ? wn / 2 : wn);
        const int out = which;
        t += per_xcd;
        const bool more = t < t_end;
        if (more) place(t);
        // Strips of 16 rows pass through LDS, so that rows are written in whole runs of 8
        // columns and the code that writes them stands here once (written out for every
        // fragment, with four activations, it does not fit the instruction cache: a tile's
        // results took 21 us). Each strip begins with an eighth of the next tile's first
        // loads. Accumulators go to LDS from their registers: lane l holds columns 16 j +
        // 4 (l >> 4) .. +3 of row l & 15; 16-byte chunk c of row r lies at c ^ (r & 7).
        float* strip = sE[wave];
        const uint32_t strip_at = (uint32_t)(uintptr_t)(LDSP float*)strip;
        const uint32_t put0 = strip_at + (lane & 15) * 512 + (((lane >> 4) ^ (lane & 7)) << 4), put1 = put0 ^ 64;
#pragma clang loop unroll(disable)
        for (int i = 0; i < F; ++i) {
            static_for<0, F>([&](auto ic) {
                constexpr int I = decltype(ic)::value;
                if (i != I) return;
                if (more) start(ic);
                static_for<0, F>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    put_acc<I, j / 2 * 128>(acc[I][j], j % 2 == 0 ? put0 : put1);
                });
            });
            // This lane's runs of the strip, 8 columns of a row each: pass p takes row p RPP +
            // lane / LPR. Read here in one piece, with its own wait: at a read that the
            // compiler sees it would wait for the next tile's loads. (A wave's LDS
            // instructions execute in order, so the writes above need none.)
            constexpr int LPR = DUAL ? 8 : 16, RPP = 64 / LPR, PASSES = 16 / RPP;
            const int r0 = lane / LPR, c = 2 * (lane % LPR);   // (c: the run's first chunk)
            f32x4 x[8];
            {
                const uint32_t base = strip_at + r0 * 512;
                const uint32_t e0 = base + ((c ^ (r0 & 7)) << 4), e1 = base + (((c + 1) ^ (r0 & 7)) << 4);
                if constexpr (DUAL) {   // rows r0 and r0 + 8, of each the gate's run and the up projection's
                    asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
                                 "ds_read_b128 %2, %8 offset:256\n\tds_read_b128 %3, %9 offset:256\n\t"
                                 "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
                                 "ds_read_b128 %6, %8 offset:4352\n\tds_read_b128 %7, %9 offset:4352\n\t"
                                 "s_waitcnt lgkmcnt(0)"
                                 : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
                                 : "v"(e0), "v"(e1)
                                 : "memory");
                } else {   // rows r0, r0 + 4, r0 + 8, r0 + 12
                    const uint32_t o0 = base + ((c ^ (r0 & 7) ^ 4) << 4), o1 = base + (((c + 1) ^ (r0 & 7) ^ 4) << 4);
                    asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
                                 "ds_read_b128 %2, %10 offset:2048\n\tds_read_b128 %3, %11 offset:2048\n\t"
                                 "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
                                 "ds_read_b128 %6, %10 offset:6144\n\tds_read_b128 %7, %11 offset:6144\n\t"
                                 "s_waitcnt lgkmcnt(0)"
                                 : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
                                 : "v"(e0), "v"(e1), "v"(o0), "v"(o1)
                                 : "memory");
                }
            }
            auto run = [&](int n, float (&v)[8]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) { v[e] = x[2 * n][e]; v[e + 4] = x[2 * n + 1][e]; }
            };
            const int64_t row1 = row0 + i * 16, col = col0 + 4 * c;
            const int cnt = (int)min((int64_t)8, A.n - col);   // columns of this run that exist
            // Rows p of a result from the strip's first on. ALIGNED (rows of whole 16-byte runs):
            // through a resource that ends with the result, at one offset a lane; else by address.
            auto rows_of = [&](void* p, int64_t ld, int es) {
                const int rows = (int)max(min(A.m - row1, (int64_t)16), (int64_t)0);
                // (nothing, where this wave's columns begin behind the last one)
                return resource((const char*)p + (row1 * ld + col0) * es, max(rows * (int)ld - (int)col0, 0) * es);
            };
            auto put = [&](bf16* p, int64_t ld, int pass, int n, const float (&v)[8]) {
                if (A.aligned) {
                    const int off = cnt > 0 ? (int)((r0 + pass * RPP) * ld + 4 * c) * 2 : OUTSIDE;
                    bf16x8 x;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = (bf16)v[e];
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), rows_of(p, ld, 2), off, 0, 0);
                } else if (row1 + r0 + pass * RPP < A.m && cnt > 0) {
                    store_run<bf16, 8>(p + (row1 + r0 + pass * RPP) * ld + col, n, v);
                }
            };
            auto put32 = [&](float* p, int64_t ld, int pass, const float (&v)[8]) {
                if (A.aligned) {
                    const int off = cnt > 0 ? (int)((r0 + pass * RPP) * ld + 4 * c) * 4 : OUTSIDE;
                    const auto rs = rows_of(p, ld, 4);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), rs, off, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}), rs, off + 16, 0, 0);
                } else if (row1 + r0 + pass * RPP < A.m && cnt > 0) {
                    store_run<float, 8>(p + (row1 + r0 + pass * RPP) * ld + col, cnt, v);
                }
            };
            if constexpr (DUAL) {
                float v[16], w[16], o[16], s[16];
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    float y[8], z[8];
                    run(2 * p, y);
                    run(2 * p + 1, z);
                    if (MODE == FWD && A.gates[0]) {
                        if (A.gates_f32) {
                            put32((float*)A.gates[0], A.ldo, p, y);
                            put32((float*)A.gates[1], A.ldo, p, z);
                        } else {
                            put((bf16*)A.gates[0], A.ldo, p, cnt, y);
                            put((bf16*)A.gates[1], A.ldo, p, cnt, z);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) { v[8 * p + e] = y[e]; w[8 * p + e] = z[e]; }
                }
                float d[PASSES][8];
                if constexpr (MODE == RECOMP) {
#pragma unroll
                    for (int p = 0; p < PASSES; ++p) {
                        const int64_t row = row1 + r0 + p * RPP;
                        load_run<bf16, 8>((const bf16*)A.dh + row * A.n + col, row < A.m ? cnt : 0, d[p]);
                    }
                    slope_run<true>(A.act, v, o, s);
                } else {
                    act_run<true>(A.act, v, o);
                }
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    float y[8], z[8];
                    if constexpr (MODE == FWD) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = o[8 * p + e] * w[8 * p + e];
                        put((bf16*)A.out[0], A.ldo, p, cnt, y);
                    } else {   // (rows padded to whole runs: zeros behind hidden, which DX reads)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            y[e] = d[p][e] * w[8 * p + e] * s[8 * p + e];
                            z[e] = d[p][e] * o[8 * p + e];
                        }
                        put((bf16*)A.out[0], A.ldo, p, 8, y);
                        put((bf16*)A.out[1], A.ldo, p, 8, z);
                    }
                }
            } else {
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    const int64_t row = row1 + r0 + p * RPP;
                    const int some = row < A.m ? cnt : 0;
                    float v[8], w[8];
                    run(p, v);
                    if (MODE == DW && A.out_f32) {
                        if (A.accumulate) {
                            load_run<float, 8>((const float*)A.out[out] + row * A.n + col, some, w);
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] += w[e];
                        }
                        put32((float*)A.out[out], A.n, p, v);
                    } else {
                        if (MODE == DW && A.accumulate) {
                            load_run<bf16, 8>((const bf16*)A.out[out] + row * A.n + col, some, w);
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] += w[e];
                        }
                        put((bf16*)A.out[out], A.n, p, cnt, v);
                    }
                }
            }
        }
        if (!more) return;
    }
}

}  // namespace

hipError_t launch_wide(int mode, const TileArgs& a, int grid, hipStream_t s) {
    switch (mode) {
        case FWD: hipLaunchKernelGGL(k_wide<FWD>, dim3(grid), dim3(NTHR), 0, s, a); break;
        case RECOMP: hipLaunchKernelGGL(k_wide<RECOMP>, dim3(grid), dim3(NTHR), 0, s, a); break;
        case DX: hipLaunchKernelGGL(k_wide<DX>, dim3(grid), dim3(NTHR), 0, s, a); break;
        default: hipLaunchKernelGGL(k_wide<DW>, dim3(grid), dim3(NTHR), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace gated
}  // namespace mu
