// Rotary positions (gfx950): the C entry point and its kernel.
//
// Pair i of a head's first `part` elements turns by the angle p f_i of its row's
// position p:
//   (a, b) -> m (a cos - b sin, b cos + a sin)
// with (a, b) elements (i, i + part / 2), or (2 i, 2 i + 1) interleaved; the
// inverse turns by -p f_i, which with the same m is also the gradient (the
// transpose of m times a rotation). Elements from `part` on are copied.
//
// Angles are float64 turns p f_i / 2 pi less their nearest whole number, so a
// position of millions keeps its angle to 2^-52 of the turns it made; sine and
// cosine of what is left are float32 (half a turn's argument is exact to 2^-25).
// They are shared by all heads: a workgroup computes those of its rows once, into
// LDS, and then streams the rows of every head of both tensors.
//
// What bounds it: HBM, every element read once and written once. 8192 rows of 32 + 8 heads
// of 128, inputs cold: bfloat16 34 to 36 us, 4.7 to 4.9 TB/s, float32 63 to 68, 5.0 to 5.3, the
// rate of a large copy. Rows of single tokens: 4.6 us for 64.
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

constexpr int NTHR = 256;
constexpr int MAX_CS = 2048;   // angles of a workgroup: 16 KB of LDS
constexpr int MAX_TOK = 64;    // rows of a workgroup

// Units of a thread, a vector of pairs or one of each half: four vectors are on their way
// before the angles are computed. Halves with two units 33.4 us, with four 36.1, one 36;
// pairs with four 34, with two 35.9 (8192 rows of 32 + 8 heads of 128, bfloat16, cold).
template <bool PAIRS> constexpr int per() { return PAIRS ? 4 : 2; }

struct RotArgs {
    mu_rotary_args a;
    int tok;         // rows of a workgroup
    int rot;         // vectors (halves: of one half) that turn, of each head
    int items;       // vectors of a row: all heads of all tensors
    int per_head;    // vectors of a head: those that turn, then those that are copied
};

template <typename T, bool PAIRS>
__global__ __launch_bounds__(NTHR) void k_rotary(RotArgs A) {
    constexpr int V = vec_of<T>(), PER = per<PAIRS>();
    typedef typename VecOf<T>::V Vec;
    __shared__ float2 cs[MAX_CS];
    const mu_rotary_args& R = A.a;
    const uint32_t half = R.part >> 1, len = (uint32_t)R.len;
    const uint32_t rows = (uint32_t)(R.batch * R.len), row0 = blockIdx.x * (uint32_t)A.tok;   // (up to 2^31)
    const uint32_t ntok = min((uint32_t)A.tok, rows - row0);

    // this thread's vectors (blockIdx.y cuts the rows' vectors): where they lie, and the loads
    const uint32_t total = ntok * A.items, first = blockIdx.y * (NTHR * PER) + threadIdx.x;
    Vec x0[PER], x1[PER];
    T* out[PER];
    int cnt[PER];
    uint32_t ang[PER];   // of its first element, or (copied) ~0
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const uint32_t i = first + j * NTHR;
        cnt[j] = 0;
        if (i >= total) continue;
        const uint32_t t = i / (uint32_t)A.items, w = i - t * A.items;
        uint32_t head = w / (uint32_t)A.per_head;
        const int v = (int)(w - head * A.per_head);
        const int which = R.n == 2 && head >= (uint32_t)R.x[0].heads ? 1 : 0;
        const mu_rotary_tensor& X = R.x[which];
        if (which) head -= R.x[0].heads;
        const uint32_t row = row0 + t, b = row / len, s = row - b * len;
        const T* x = (const T*)X.x + (int64_t)b * X.x_stride_b + (int64_t)s * X.x_stride_s + (int64_t)head * X.x_stride_h;
        T* o = (T*)X.out + (int64_t)b * X.out_stride_b + (int64_t)s * X.out_stride_s + (int64_t)head * X.out_stride_h;
        int e0 = v * V;
        ang[j] = t * half + (PAIRS ? e0 / 2 : e0);
        cnt[j] = min(V, (PAIRS ? R.part : (int)half) - e0);
        if (v >= A.rot) {   // behind the part that turns
            e0 = R.part + (v - A.rot) * V;
            ang[j] = ~0u;
            cnt[j] = min(V, R.dim - e0);
        }
        out[j] = o + e0;
        x0[j] = load_vec<T>(x + e0, cnt[j]);
        if (!PAIRS && ang[j] != ~0u) x1[j] = load_vec<T>(x + half + e0, cnt[j]);
    }

    for (uint32_t i = threadIdx.x; i < ntok * half; i += NTHR) {
        const uint32_t t = i / half, f = i - t * half;
        const uint32_t row = row0 + t, s = row % len;
        int64_t p = R.offset;
        if (R.positions) {
            const uint32_t at = R.shared_positions ? s : row;
            p += R.position_bits == 32 ? (int64_t)gp((const int32_t*)R.positions)[at] : gp((const int64_t*)R.positions)[at];
        } else {
            p += s;
        }
        const double turns = (double)p * (gp(R.freqs)[f] * 0.15915494309189535);   // 1 / 2 pi
        const float half_turns = (float)(2.0 * (turns - rint(turns)));
        float sn, c;
        sincospif(half_turns, &sn, &c);
        cs[i] = make_float2(c * R.scale, (R.inverse ? -sn : sn) * R.scale);
    }
    __syncthreads();

#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (cnt[j] <= 0) continue;
        if (ang[j] != ~0u) {
#pragma unroll
            for (int e = 0; e < V; e += PAIRS ? 2 : 1) {
                const float2 q = cs[min(ang[j] + (PAIRS ? e / 2 : e), (uint32_t)MAX_CS - 1)];   // (behind cnt: any)
                const float a = to_f32<T>(x0[j][e]), c = PAIRS ? to_f32<T>(x0[j][e + (PAIRS ? 1 : 0)]) : to_f32<T>(x1[j][e]);
                x0[j][e] = from_f32<T>(a * q.x - c * q.y);
                if (PAIRS) x0[j][e + (PAIRS ? 1 : 0)] = from_f32<T>(c * q.x + a * q.y);
                else x1[j][e] = from_f32<T>(c * q.x + a * q.y);
            }
            if (!PAIRS) store_vec<T>(out[j] + half, cnt[j], x1[j]);
        }
        store_vec<T>(out[j], cnt[j], x0[j]);
    }
}

size_t es_of(int dtype) { return dtype == MU_BF16 ? 2 : 4; }

// One strided view [batch, len, heads, dim] of elements.
struct View {
    const void* p;
    int64_t sb, ss, sh;
    int64_t batch, len, heads, dim;
    size_t es;
    int64_t row() const { return (heads - 1) * sh + dim; }   // elements from a row's first to its last
    bool empty() const { return batch == 0 || len == 0 || heads == 0; }
    uintptr_t lo() const { return (uintptr_t)p; }
    uintptr_t hi() const { return lo() + (size_t)((batch - 1) * sb + (len - 1) * ss + row()) * es; }
    bool same(const View& o) const {
        return p == o.p && heads == o.heads && (batch == 1 || sb == o.sb) && (len == 1 || ss == o.ss) && (heads == 1 || sh == o.sh);
    }
    bool sane() const {
        const double n = (double)(batch - 1) * (double)sb + (double)(len - 1) * (double)ss + (double)(heads - 1) * (double)sh + (double)dim;
        return n <= (double)((int64_t)1 << 50);
    }
    // every element has an address of its own: strides nest
    bool distinct() const {
        struct { int64_t n, s; } d[3] = {{batch, sb}, {len, ss}, {heads, sh}};
        std::sort(d, d + 3, [](auto& x, auto& y) { return x.s < y.s; });
        int64_t extent = dim;
        for (auto& x : d) {
            if (x.n <= 1) continue;
            if (x.s < extent) return false;
            extent += (x.n - 1) * x.s;
        }
        return true;
    }
};

// Whether delta + sum of x[i] * s[i] + e = 0 has a solution in whole numbers lo[i] <= x[i] <= hi[i]
// and |e| < dim: whether two views of the same strides share an element, x being the differences
// of their indices. Strides descend; where they nest at most two x of each are in reach of the
// strides behind it. `left` bounds the search for any others, which then counts as a yes.
struct Steps {
    int64_t s[3], lo[3], hi[3];
    int n;
};
bool meet(const Steps& t, int i, int64_t delta, int64_t dim, int& left) {
    if (i == t.n) return delta > -dim && delta < dim;
    int64_t reach = dim - 1;
    for (int j = i + 1; j < t.n; ++j) reach += t.s[j] * std::max(-t.lo[j], t.hi[j]);
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); };
    const int64_t lo = std::max(t.lo[i], -floor_div(delta + reach, t.s[i])), hi = std::min(t.hi[i], floor_div(reach - delta, t.s[i]));
    for (int64_t x = lo; x <= hi; ++x)
        if (--left < 0 || meet(t, i + 1, delta + x * t.s[i], dim, left)) return true;
    return false;
}

// Views that share no element: apart in memory, of the same strides (of sizes above one) with
// no element in common, or column ranges of rows of one pitch.
bool apart(View a, View b) {
    if (a.empty() || b.empty() || a.hi() <= b.lo() || b.hi() <= a.lo()) return true;
    const struct { int64_t na, nb, sa, sb; } d[3] = {{a.batch, b.batch, a.sb, b.sb}, {a.len, b.len, a.ss, b.ss}, {a.heads, b.heads, a.sh, b.sh}};
    Steps t{{}, {}, {}, 0};
    bool alike = true;
    for (const auto& x : d) {
        if (x.na == 1 && x.nb == 1) continue;
        if (x.na > 1 && x.nb > 1 && x.sa != x.sb) alike = false;
        const int64_t s = x.na > 1 ? x.sa : x.sb;
        if (s == 0) continue;   // (an input's: one element for all indices)
        int i = t.n++;
        for (; i > 0 && t.s[i - 1] < s; --i) {
            t.s[i] = t.s[i - 1];
            t.lo[i] = t.lo[i - 1];
            t.hi[i] = t.hi[i - 1];
        }
        t.s[i] = s;
        t.lo[i] = 1 - x.na;
        t.hi[i] = x.nb - 1;
    }
    int left = 64;
    if (alike) return !meet(t, 0, ((int64_t)b.lo() - (int64_t)a.lo()) / (int64_t)a.es, a.dim, left);
    if (a.lo() > b.lo()) std::swap(a, b);
    for (View* v : {&a, &b})
        if (v->len == 1) { v->len = v->batch; v->ss = v->sb; v->batch = 1; }
    if (a.ss != b.ss || a.ss <= 0 || a.len == 1) return false;
    if ((a.batch > 1 && a.sb % a.ss != 0) || (b.batch > 1 && b.sb % b.ss != 0)) return false;
    const int64_t pitch = a.ss * (int64_t)a.es, ra = a.row() * (int64_t)a.es, rb = b.row() * (int64_t)b.es;
    const int64_t c = (int64_t)((b.lo() - a.lo()) % pitch);   // b's first column behind a's
    return c >= ra && c + rb <= pitch;
}

int check(const mu_rotary_args* a) {
    if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
    if (a->dtype != MU_F32 && a->dtype != MU_BF16) return fail(MU_ERR_DTYPE, "unknown dtype %d", a->dtype);
    if (a->n < 1 || a->n > 2) return fail(MU_ERR_INVALID_ARG, "n must be 1 or 2");
    if (a->batch < 0 || a->len < 0 || a->batch > 0x7fffffffLL || a->len > 0x7fffffffLL ||
        (a->len > 0 && a->batch > 0x7fffffffLL / a->len))
        return fail(MU_ERR_INVALID_ARG, "bad batch or length");
    if (a->dim < 1 || a->dim > MU_ROTARY_MAX_DIM) return fail(MU_ERR_INVALID_ARG, "dim must be in [1, %d]", MU_ROTARY_MAX_DIM);
    if (a->part < 2 || a->part > a->dim || a->part % 2 != 0) return fail(MU_ERR_INVALID_ARG, "part must be even and in [2, dim]");
    for (int flag : {a->interleaved, a->inverse, a->shared_positions})
        if (flag != 0 && flag != 1) return fail(MU_ERR_INVALID_ARG, "interleaved, inverse and shared_positions must be 0 or 1");
    if (!std::isfinite(a->scale)) return fail(MU_ERR_INVALID_ARG, "scale must be finite");
    if (a->offset < -((int64_t)1 << 52) || a->offset > ((int64_t)1 << 52)) return fail(MU_ERR_INVALID_ARG, "offset is too large");
    if (a->positions && a->position_bits != 32 && a->position_bits != 64)
        return fail(MU_ERR_DTYPE, "positions must be int32 or int64 (position_bits %d)", a->position_bits);
    if (!a->freqs) return fail(MU_ERR_INVALID_ARG, "freqs is null");
    if (!aligned(a->freqs, 8) || (a->positions && !aligned(a->positions, a->position_bits / 8)))
        return fail(MU_ERR_LAYOUT, "misaligned freqs or positions");
    const size_t es = es_of(a->dtype);
    std::vector<View> in, out;
    for (int i = 0; i < a->n; ++i) {
        const mu_rotary_tensor& t = a->x[i];
        if (t.heads < 0 || t.heads > (1 << 16)) return fail(MU_ERR_INVALID_ARG, "tensor %d: bad head count", i);
        for (int64_t s : {t.x_stride_b, t.x_stride_s, t.x_stride_h, t.out_stride_b, t.out_stride_s, t.out_stride_h})
            if (s < 0) return fail(MU_ERR_INVALID_ARG, "tensor %d: strides must be >= 0", i);
        if (a->batch == 0 || a->len == 0 || t.heads == 0) continue;
        if (!t.x || !t.out) return fail(MU_ERR_INVALID_ARG, "tensor %d: null x or out", i);
        if (!aligned(t.x, es) || !aligned(t.out, es)) return fail(MU_ERR_LAYOUT, "tensor %d: misaligned buffer", i);
        in.push_back({t.x, t.x_stride_b, t.x_stride_s, t.x_stride_h, a->batch, a->len, t.heads, a->dim, es});
        out.push_back({t.out, t.out_stride_b, t.out_stride_s, t.out_stride_h, a->batch, a->len, t.heads, a->dim, es});
        if (!in.back().sane() || !out.back().sane()) return fail(MU_ERR_INVALID_ARG, "tensor %d: strides are too large", i);
        if (!out.back().distinct()) return fail(MU_ERR_LAYOUT, "tensor %d: out overlaps itself", i);
    }
    for (size_t i = 0; i < out.size(); ++i) {
        for (size_t j = 0; j < in.size(); ++j) {
            if (!apart(out[i], in[j]) && !(i == j && out[i].same(in[j])))
                return fail(MU_ERR_LAYOUT, "out overlaps an input that is not the same tensor");
            if (j > i && !apart(out[i], out[j])) return fail(MU_ERR_LAYOUT, "outputs overlap");
        }
        const int64_t np = a->shared_positions ? a->len : a->batch * a->len;
        const uintptr_t f = (uintptr_t)a->freqs, p = (uintptr_t)a->positions;
        if ((out[i].lo() < f + 4 * (size_t)a->part && f < out[i].hi()) ||
            (p && out[i].lo() < p + (size_t)np * (a->position_bits / 8) && p < out[i].hi()))
            return fail(MU_ERR_LAYOUT, "out overlaps freqs or positions");
    }
    return MU_OK;
}

template <typename T>
hipError_t launch(const RotArgs& r, dim3 grid, hipStream_t s) {
    if (r.a.interleaved) hipLaunchKernelGGL((k_rotary<T, true>), grid, dim3(NTHR), 0, s, r);
    else hipLaunchKernelGGL((k_rotary<T, false>), grid, dim3(NTHR), 0, s, r);
    return hipGetLastError();
}

}  // namespace

extern "C" {

int mu_rotary(const mu_rotary_args* a, void* stream) {
    return guarded([&]() -> int {
        int rc = check(a);
        if (rc) return rc;
        const int64_t rows = a->batch * a->len, heads = (int64_t)a->x[0].heads + (a->n == 2 ? a->x[1].heads : 0);
        if (rows == 0 || heads == 0) return MU_OK;
        const size_t es = es_of(a->dtype);
        const int v = (int)(16 / es), turning = a->interleaved ? a->part : a->part / 2;
        // in place the rest of each head stays where it is
        bool in_place = true;
        for (int i = 0; i < a->n; ++i) in_place = in_place && (a->x[i].heads == 0 || a->x[i].x == a->x[i].out);
        RotArgs r{*a, 0, 0, 0, 0};
        r.rot = (turning + v - 1) / v;
        r.per_head = r.rot + (in_place ? 0 : (a->dim - a->part + v - 1) / v);
        if (heads * r.per_head > (1 << 24)) return fail(MU_ERR_INVALID_ARG, "too many elements in a row");
        r.items = (int)heads * r.per_head;
        // as many rows as fill a workgroup's threads `per` times, their angles within LDS; few
        // rows: as many as fill them once, a long row's heads shared out over workgroups
        const int PER = a->interleaved ? per<true>() : per<false>();
        const int64_t few = rows * r.items <= 256 * NTHR * PER ? 1 : PER;
        r.tok = (int)std::max<int64_t>(1, std::min<int64_t>({MAX_TOK, MAX_CS / (a->part / 2), few * NTHR / r.items, rows}));
        const int64_t wgs = (rows + r.tok - 1) / r.tok;
        const int ny = (r.tok * r.items + NTHR * PER - 1) / (NTHR * PER);
        if (wgs > 0xffffffffLL / NTHR || ny > 65535) return fail(MU_ERR_INVALID_ARG, "too many rows for one launch at this size");
        const double cells = (double)rows * (double)heads;
        const double bytes = cells * 2.0 * (in_place ? a->part : a->dim) * (double)es + (a->positions ? rows * (a->position_bits / 8.0) : 0.0);
        hipStream_t s = (hipStream_t)stream;
        return timed_launch(MU_K_ROTARY, 3.0 * cells * a->part, bytes, s, [&] {
            const dim3 grid((unsigned)wgs, (unsigned)ny);
            return a->dtype == MU_BF16 ? launch<bf16>(r, grid, s) : launch<float>(r, grid, s);
        }, "rotary launch");
    });
}

}  // extern "C"
