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
// What bounds it: HBM, every element read once and written once.
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

struct RotArgs {
    mu_rotary_args a;
    int tok;         // rows of a workgroup
    int rot;         // vectors (halves: of one half) that turn, of each head
    int items;       // vectors of a row: all heads of all tensors
    int per_head;    // vectors of a head: those that turn, then those that are copied
    int chunk;       // vectors of a workgroup (blockIdx.y cuts the rows' vectors)
};

template <typename T, bool PAIRS>
__global__ __launch_bounds__(NTHR) void k_rotary(RotArgs A) {
    constexpr int V = vec_of<T>();
    __shared__ float2 cs[MAX_CS];
    const mu_rotary_args& R = A.a;
    const int half = R.part >> 1;
    const int64_t rows = R.batch * R.len, row0 = (int64_t)blockIdx.x * A.tok;
    const int ntok = (int)min((int64_t)A.tok, rows - row0);

    for (int i = threadIdx.x; i < ntok * half; i += NTHR) {
        const int t = i / half, f = i - t * half;
        const int64_t row = row0 + t, s = row % R.len;
        int64_t p = R.offset;
        if (R.positions) {
            const int64_t at = R.shared_positions ? s : row;
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

    const int total = ntok * A.items, first = blockIdx.y * A.chunk, last = min(total, first + A.chunk);
    for (int i = first + threadIdx.x; i < last; i += NTHR) {
        const int t = i / A.items, w = i - t * A.items;
        int head = w / A.per_head;
        const int v = w - head * A.per_head;
        const int which = R.n == 2 && head >= R.x[0].heads ? 1 : 0;
        const mu_rotary_tensor& X = R.x[which];
        if (which) head -= R.x[0].heads;
        const int64_t row = row0 + t, b = row / R.len, s = row - b * R.len;
        const T* x = (const T*)X.x + b * X.x_stride_b + s * X.x_stride_s + head * X.x_stride_h;
        T* o = (T*)X.out + b * X.out_stride_b + s * X.out_stride_s + head * X.out_stride_h;
        const float2* ang = cs + t * half;
        if (v >= A.rot) {   // behind the part that turns: the same bits
            const int e0 = R.part + (v - A.rot) * V, cnt = min(V, R.dim - e0);
            if (cnt == V) *(MU_GLOBAL typename VecOf<T>::U*)gp(o + e0) = *(const MU_GLOBAL typename VecOf<T>::U*)gp(x + e0);
            else
                for (int e = 0; e < cnt; ++e) gp(o)[e0 + e] = gp(x)[e0 + e];
        } else if constexpr (PAIRS) {
            const int e0 = v * V, cnt = min(V, R.part - e0);
            float y[V];
            load_run<T, V>(x + e0, cnt, y);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float2 q = ang[min((e0 + e) >> 1, half - 1)];
                const float a = y[e], c = y[e + 1];
                y[e] = a * q.x - c * q.y;
                y[e + 1] = c * q.x + a * q.y;
            }
            store_run<T, V>(o + e0, cnt, y);
        } else {
            const int e0 = v * V, cnt = min(V, half - e0);
            float y[V], z[V];
            load_run<T, V>(x + e0, cnt, y);
            load_run<T, V>(x + half + e0, cnt, z);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 q = ang[min(e0 + e, half - 1)];
                const float a = y[e], c = z[e];
                y[e] = a * q.x - c * q.y;
                z[e] = c * q.x + a * q.y;
            }
            store_run<T, V>(o + e0, cnt, y);
            store_run<T, V>(o + half + e0, cnt, z);
        }
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

// Views that share no element: apart in memory, or column ranges of rows of one pitch.
bool apart(View a, View b) {
    if (a.empty() || b.empty() || a.hi() <= b.lo() || b.hi() <= a.lo()) return true;
    if (a.lo() > b.lo()) std::swap(a, b);
    for (View* v : {&a, &b})
        if (v->len == 1) { v->len = v->batch; v->ss = v->sb; v->batch = 1; }
    if (a.ss != b.ss || a.ss <= 0 || a.len == 1) return false;
    if ((a.batch > 1 && a.sb % a.ss != 0) || (b.batch > 1 && b.sb % b.ss != 0)) return false;
    const int64_t pitch = a.ss * (int64_t)a.es, ra = a.row() * (int64_t)a.es, rb = b.row() * (int64_t)b.es;
    const int64_t d = (int64_t)((b.lo() - a.lo()) % pitch);   // b's first column behind a's
    return d >= ra && d + rb <= pitch;
}

int check(const mu_rotary_args* a) {
    if (!a) return fail(MU_ERR_INVALID_ARG, "argument is null");
    if (a->dtype != MU_F32 && a->dtype != MU_BF16) return fail(MU_ERR_DTYPE, "unknown dtype %d", a->dtype);
    if (a->n < 1 || a->n > 2) return fail(MU_ERR_INVALID_ARG, "n must be 1 or 2");
    if (a->batch < 0 || a->len < 0 || a->batch > ((int64_t)1 << 31) || a->len > ((int64_t)1 << 31) ||
        (a->len > 0 && a->batch > ((int64_t)1 << 31) / a->len))
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
        RotArgs r{*a, 0, 0, 0, 0, 0};
        r.rot = (turning + v - 1) / v;
        r.per_head = r.rot + (in_place ? 0 : (a->dim - a->part + v - 1) / v);
        if (heads * r.per_head > (1 << 24)) return fail(MU_ERR_INVALID_ARG, "too many elements in a row");
        r.items = (int)heads * r.per_head;
        // some four vectors a thread, the angles of the rows within LDS
        r.tok = std::max(1, std::min({MAX_TOK, MAX_CS / (a->part / 2), 4 * NTHR / r.items}));
        r.tok = (int)std::min<int64_t>(r.tok, rows);
        const int64_t wgs = (rows + r.tok - 1) / r.tok;
        if (wgs > 0xffffffffLL / NTHR) return fail(MU_ERR_INVALID_ARG, "too many rows for one launch at this size");
        // few rows: their heads are shared out over workgroups, a vector a thread
        const int total = r.tok * r.items;
        const int cuts = (int)std::max<int64_t>(1, std::min<int64_t>({(total + NTHR - 1) / NTHR, 512 / wgs, 65535}));
        r.chunk = ((total + cuts - 1) / cuts + NTHR - 1) / NTHR * NTHR;
        const int ny = (total + r.chunk - 1) / r.chunk;
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
