// Rotary positions of q and k with one to four position axes (fl_rope).
//
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),
//   t = positions[axis_of[i]][row] * inv_freq[i]
//
// Bound by HBM: every channel is read and written once. The angle depends on
// the row and the pair only, so a CTA computes the sines of its rows once into
// shared memory and applies them to every head of q and k; a thread has four
// tasks (8 pairs of a head each, two 16-byte vectors) in flight, the first of
// them requested before the sines are computed. Measured in graphs: 4099 rows of 32 and 8
// heads of 128 on three axes 14.9 us (5.6 TB/s); 7 rows 2.2 us, a launch and one
// round trip for the positions and one for the vectors.
//
// The angle is taken in turns, in fixed point: f = frac(inv_freq / 2 pi) as a
// 64-bit fraction, from the 24-bit significand of inv_freq times 64 bits of
// 1 / 2 pi, and position * f modulo 2^64 is the fraction of a turn, exact in
// the position: for the largest int32 position and a frequency up to 256 the
// error is below 2^-24 turns, where the fp32 product position * inv_freq would
// be off by whole turns. The top 32 bits go to sincospif.
#include "fl_common.cuh"
#include "fl_host.h"

namespace fl {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;  // rows of one CTA at most
constexpr int kRopePairs = FL_ROPE_MAX_DIM / 2;
constexpr int kMaxHeads = 4096;

struct RopeParams {
    const uint16_t* x[2];  // q, k
    uint16_t* y[2];
    long long x_row[2], x_head[2], y_row[2], y_head[2];
    const int* positions;
    const float* inv_freq;
    long long positions_stride;
    int rows, heads[2], head_dim, pairs, rows_per_cta;
    uint32_t per, per_inv;      // tasks of a head's row, and 2^32 / it rounded up
    uint32_t all, all_inv;      // heads of q and k, likewise
    uint32_t pairs_inv;
    int interleaved, inverse;
    int copy;  // channels behind the rotated ones are copied (out of place)
    unsigned char axis_of[kRopePairs];
};

// n / d with inv = ceil(2^32 / d): exact while n * d < 2^32 (here n is at most 4 rows * kMaxHeads * d, d at most 512).
__device__ __forceinline__ uint32_t quick_div(uint32_t n, uint32_t d, uint32_t inv) { return d == 1 ? n : __umulhi(n, inv); }

// frac(f / 2 pi) in units of 2^-64 turns: f = m 2^e with a 24-bit integer m, and
// 1 / 2 pi = kInv 2^-66 (64 bits of it), so the fraction is m kInv 2^(e - 2)
// modulo 2^64.
__device__ __forceinline__ unsigned long long turns_per_position(float f) {
    constexpr unsigned long long kInv = 0xa2f9836e4e441529ull;  // 2^66 / (2 pi), rounded down
    const uint32_t u = __float_as_uint(f), x = (u >> 23) & 255u;
    const unsigned long long m = (u & 0x7fffffu) | (x != 0u ? 0x800000u : 0u);
    const int e = (int)(x != 0u ? x : 1u) - 150 - 2;  // power of the last place of m * kInv, in units of 2^-64
    const unsigned long long lo = m * kInv, hi = __umul64hi(m, kInv);
    unsigned long long t;
    if (e >= 0)
        t = e < 64 ? lo << e : 0ull;
    else if (e > -64)
        t = (lo >> -e) | (hi << (64 + e));
    else
        t = e > -128 ? hi >> (-e - 64) : 0ull;
    return u >> 31 ? 0ull - t : t;
}

template <int DT>
__device__ __forceinline__ void rotate2(uint32_t a, uint32_t b, float2 cs0, float2 cs1, uint32_t& oa, uint32_t& ob) {
    using Ops = DTypeOps<DT>;
    const float2 x = Ops::unpack(a), y = Ops::unpack(b);
    oa = Ops::pack(fmaf(x.x, cs0.x, -y.x * cs0.y), fmaf(x.y, cs1.x, -y.y * cs1.y));
    ob = Ops::pack(fmaf(y.x, cs0.x, x.x * cs0.y), fmaf(y.y, cs1.x, x.y * cs1.y));
}

// VEC: 8 (16-byte vectors, everything aligned to them) or 1.
template <int DT, int VEC>
__global__ void __launch_bounds__(kRopeThreads) fl_rope_kernel(const __grid_constant__ RopeParams p) {
    using Ops = DTypeOps<DT>;
    // (cos, sin) of the rows' pairs. In the vector form a thread reads 8
    // neighbouring pairs as four float4, and its neighbours the next 8: the
    // first float4 of every 8 lie side by side, then the second ones, ..
    __shared__ __align__(16) float2 cs[kRopeRows][kRopePairs];
    const int r0 = blockIdx.x * p.rows_per_cta, nr = min(p.rows_per_cta, p.rows - r0);
    const uint32_t rot = (uint32_t)p.pairs / VEC, tasks = (uint32_t)nr * p.all * p.per;
    constexpr int U = VEC == 8 ? 4 : 1;  // tasks in flight per thread
    // one task: VEC pairs of one head's row, or VEC channels behind them
    struct Task {
        const uint16_t* x;
        uint16_t* y;
        int r, i, ia, ib;  // ib < 0: channels that are copied
    };
    auto task = [&](uint32_t t) {
        const uint32_t hr = quick_div(t, p.per, p.per_inv), u = t - hr * p.per;
        const uint32_t r = quick_div(hr, p.all, p.all_inv);
        const int h2 = (int)(hr - r * p.all), w = h2 >= p.heads[0], h = w ? h2 - p.heads[0] : h2;
        Task k;
        k.x = p.x[w] + (r0 + (long long)r) * p.x_row[w] + h * p.x_head[w];
        k.y = p.y[w] + (r0 + (long long)r) * p.y_row[w] + h * p.y_head[w];
        k.r = (int)r;
        k.i = (int)u * VEC;
        if (u < rot) {
            k.ia = p.interleaved ? 2 * k.i : k.i;
            k.ib = p.interleaved ? 2 * k.i + VEC : k.i + p.pairs;
        } else {
            k.ia = 2 * p.pairs + (int)(u - rot) * VEC;
            k.ib = -1;
        }
        return k;
    };
    griddep_wait();
    griddep_launch_dependents();
    uint4 a[U], b[U];
    uint16_t sa = 0, sb = 0;
    auto load = [&](uint32_t t0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t t = t0 + j * kRopeThreads;
            if (t >= tasks) continue;
            const Task k = task(t);
            if constexpr (VEC == 8) {
                a[j] = *reinterpret_cast<const uint4*>(k.x + k.ia);
                if (k.ib >= 0) b[j] = *reinterpret_cast<const uint4*>(k.x + k.ib);
            } else {
                sa = k.x[k.ia];
                if (k.ib >= 0) sb = k.x[k.ib];
            }
        }
    };
    load(threadIdx.x);
    for (uint32_t e = threadIdx.x; e < (uint32_t)(nr * p.pairs); e += kRopeThreads) {
        const uint32_t r = quick_div(e, (uint32_t)p.pairs, p.pairs_inv), i = e - r * (uint32_t)p.pairs;
        const int pos = __ldg(p.positions + p.axis_of[i] * p.positions_stride + r0 + r);
        const unsigned long long t = (unsigned long long)(long long)pos * turns_per_position(__ldg(p.inv_freq + i));
        float s, c;
        sincospif((float)(int)(t >> 32) * 0x1p-31f, &s, &c);
        cs[r][VEC == 8 ? ((i % 8 / 2) * rot + i / 8) * 2 + i % 2 : i] = make_float2(c, p.inverse ? -s : s);
    }
    __syncthreads();
    for (uint32_t t0 = threadIdx.x; t0 < tasks; t0 += U * kRopeThreads) {
        if (t0 != threadIdx.x) load(t0);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t t = t0 + j * kRopeThreads;
            if (t >= tasks) continue;
            const Task k = task(t);
            if constexpr (VEC == 8) {
                uint4 oa = a[j], ob = b[j];
                if (k.ib >= 0) {
                    const float4* f = reinterpret_cast<const float4*>(&cs[k.r][0]) + k.i / 8;
                    const uint32_t aw[4] = {a[j].x, a[j].y, a[j].z, a[j].w}, bw[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 f2 = f[e * rot];
                        if (p.interleaved) {
                            // a pair is the two halves of one word
                            const float2 v = Ops::unpack(e < 2 ? aw[2 * e] : bw[2 * e - 4]);
                            const float2 u = Ops::unpack(e < 2 ? aw[2 * e + 1] : bw[2 * e - 3]);
                            o[2 * e] = Ops::pack(fmaf(v.x, f2.x, -v.y * f2.y), fmaf(v.y, f2.x, v.x * f2.y));
                            o[2 * e + 1] = Ops::pack(fmaf(u.x, f2.z, -u.y * f2.w), fmaf(u.y, f2.z, u.x * f2.w));
                        } else {
                            rotate2<DT>(aw[e], bw[e], make_float2(f2.x, f2.y), make_float2(f2.z, f2.w), o[e], o[4 + e]);
                        }
                    }
                    oa = make_uint4(o[0], o[1], o[2], o[3]);
                    ob = make_uint4(o[4], o[5], o[6], o[7]);
                }
                *reinterpret_cast<uint4*>(k.y + k.ia) = oa;
                if (k.ib >= 0) *reinterpret_cast<uint4*>(k.y + k.ib) = ob;
            } else if (k.ib < 0) {
                k.y[k.ia] = sa;
            } else {
                const float x = Ops::unpack(sa).x, y = Ops::unpack(sb).x;
                const float2 f = cs[k.r][k.i];
                const uint32_t o = Ops::pack(fmaf(x, f.x, -y * f.y), fmaf(y, f.x, x * f.y));
                k.y[k.ia] = (uint16_t)(o & 0xffffu);
                k.y[k.ib] = (uint16_t)(o >> 16);
            }
        }
    }
}

struct View {
    const void* p;
    long long row, head;
    int heads;
};

size_t span(const View& v, int rows, int dim) {
    return ((size_t)(rows - 1) * v.row + (size_t)(v.heads - 1) * v.head + dim) * 2;
}

}  // namespace

}  // namespace fl

namespace fl {
namespace {

// The checks of fl_rope, and its launch unless `check_only`.
fl_status rope(const fl_rope_desc* d, bool check_only, cudaStream_t s) {
    using host::fail;
    if (d == nullptr) return fail(FL_ERR_INVALID_ARG, "fl_rope: null description");
    if (!host::valid_dtype(d->dtype)) return fail(FL_ERR_INVALID_ARG, "fl_rope: bad dtype %d", (int)d->dtype);
    if (d->rows < 0 || d->heads_q < 1 || d->heads_k < 0 || d->head_dim < 1)
        return fail(FL_ERR_INVALID_ARG, "fl_rope: sizes must be positive (rows may be 0)");
    if (d->heads_q + (long long)d->heads_k > kMaxHeads)
        return fail(FL_ERR_UNSUPPORTED, "fl_rope: more than %d heads of q and k", kMaxHeads);
    if (d->head_dim > FL_ROPE_MAX_DIM)
        return fail(FL_ERR_UNSUPPORTED, "fl_rope: head_dim above %d (%d)", FL_ROPE_MAX_DIM, d->head_dim);
    if (d->rotary_dim < 2 || d->rotary_dim % 2 != 0 || d->rotary_dim > d->head_dim)
        return fail(FL_ERR_INVALID_ARG, "fl_rope: rotary_dim must be even, 2 .. head_dim (%d of %d)", d->rotary_dim,
                    d->head_dim);
    if (d->n_axes < 1 || d->n_axes > 4) return fail(FL_ERR_INVALID_ARG, "fl_rope: n_axes must be 1 .. 4 (%d)", d->n_axes);
    const int pairs = d->rotary_dim / 2;
    for (int i = 0; d->axis_of != nullptr && i < pairs; ++i)
        if (d->axis_of[i] >= d->n_axes)
            return fail(FL_ERR_INVALID_ARG, "fl_rope: pair %d takes axis %d of %d", i, (int)d->axis_of[i], d->n_axes);
    if (d->rows == 0) return host::ok();
    const bool has_k = d->heads_k > 0;
    if (d->positions == nullptr || d->inv_freq == nullptr || d->q == nullptr || d->q_out == nullptr ||
        (has_k && (d->k == nullptr || d->k_out == nullptr)))
        return fail(FL_ERR_INVALID_ARG, "fl_rope: a required pointer is null");
    if ((reinterpret_cast<uintptr_t>(d->positions) | reinterpret_cast<uintptr_t>(d->inv_freq)) & 3u)
        return fail(FL_ERR_ALIGNMENT, "fl_rope: positions and inv_freq must be 4-byte aligned");
    if (d->n_axes > 1 && d->positions_stride != 0 && d->positions_stride < d->rows)
        return fail(FL_ERR_INVALID_ARG, "fl_rope: positions_stride below rows (and not 0)");
    const View in[2] = {{d->q, d->q_row, d->q_head, d->heads_q}, {d->k, d->k_row, d->k_head, d->heads_k}};
    const View out[2] = {{d->q_out, d->q_out_row, d->q_out_head, d->heads_q},
                         {d->k_out, d->k_out_row, d->k_out_head, d->heads_k}};
    const int n = has_k ? 2 : 1;
    bool vec = pairs % 8 == 0 && d->head_dim % 8 == 0, in_place = true;
    for (int i = 0; i < n; ++i) {
        for (const View& v : {in[i], out[i]}) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(v.p);
            if (a & 1u) return fail(FL_ERR_ALIGNMENT, "fl_rope: tensors must be 2-byte aligned");
            if (v.row < 0 || v.head < 0) return fail(FL_ERR_INVALID_ARG, "fl_rope: negative stride");
            vec = vec && (a & 15u) == 0 && v.row % 8 == 0 && v.head % 8 == 0;
        }
        // no two elements of an output share a place
        const View& o = out[i];
        const long long by_row = (o.heads - 1) * o.head + d->head_dim, by_head = (d->rows - 1) * o.row + d->head_dim;
        if ((o.heads > 1 && o.head < d->head_dim) || (d->rows > 1 && o.row < d->head_dim) ||
            (d->rows > 1 && o.heads > 1 && o.row < by_row && o.head < by_head))
            return fail(FL_ERR_INVALID_ARG, "fl_rope: an output's strides make its rows overlap");
        const bool same = o.p == in[i].p && o.row == in[i].row && o.head == in[i].head;
        in_place = in_place && same;
        // against every input, and the other output
        for (int j = 0; j < 2 * n; ++j) {
            const View& v = j < n ? in[j] : out[j - n];
            if ((j == i && same) || j - n == i) continue;
            const long long wo = by_row, wv = (v.heads - 1) * v.head + d->head_dim;
            if (host::overlap(o.p, span(o, d->rows, d->head_dim), v.p, span(v, d->rows, d->head_dim)) &&
                !host::apart(o.p, o.row, wo, v.p, v.row, wv, 2))
                return fail(FL_ERR_INVALID_ARG, "fl_rope: an output overlaps another tensor of the call");
        }
        const size_t pos = ((size_t)(d->n_axes - 1) * d->positions_stride + d->rows) * 4;
        if (host::overlap(o.p, span(o, d->rows, d->head_dim), d->positions, pos) ||
            host::overlap(o.p, span(o, d->rows, d->head_dim), d->inv_freq, (size_t)pairs * 4))
            return fail(FL_ERR_INVALID_ARG, "fl_rope: an output overlaps another tensor of the call");
    }
    if (check_only) return host::ok();
    host::LaunchContext ctx;
    const fl_status st = host::launch_context(s, &ctx);
    if (st != FL_OK) return st;
    RopeParams p = {};
    for (int i = 0; i < n; ++i) {
        p.x[i] = static_cast<const uint16_t*>(in[i].p);
        p.y[i] = static_cast<uint16_t*>(const_cast<void*>(out[i].p));
        p.x_row[i] = in[i].row, p.x_head[i] = in[i].head;
        p.y_row[i] = out[i].row, p.y_head[i] = out[i].head;
        p.heads[i] = in[i].heads;
    }
    p.positions = d->positions, p.positions_stride = d->positions_stride, p.inv_freq = d->inv_freq;
    p.rows = d->rows, p.head_dim = d->head_dim, p.pairs = pairs;
    p.interleaved = d->interleaved != 0, p.inverse = d->inverse != 0;
    p.copy = !in_place && d->rotary_dim < d->head_dim;
    for (int i = 0; i < pairs; ++i) p.axis_of[i] = d->axis_of != nullptr ? d->axis_of[i] : 0;
    p.per = (uint32_t)(vec ? pairs / 8 : pairs) + (p.copy ? (uint32_t)(d->head_dim - d->rotary_dim) / (vec ? 8 : 1) : 0u);
    p.all = (uint32_t)(d->heads_q + (has_k ? d->heads_k : 0));
    auto inverse = [](uint32_t n) { return (uint32_t)(((1ull << 32) + n - 1) / n); };
    p.per_inv = inverse(p.per), p.all_inv = inverse(p.all), p.pairs_inv = inverse((uint32_t)pairs);
    // one row per CTA until that fills the SMs several times over
    p.rows_per_cta = 1;
    auto ctas = [&] { return ((long long)d->rows + p.rows_per_cta - 1) / p.rows_per_cta; };
    while (p.rows_per_cta < kRopeRows && ctas() > 8 * ctx.sms) p.rows_per_cta *= 2;
    const dim3 grid((unsigned)ctas());
    cudaError_t e;
    if (d->dtype == FL_F16)
        e = vec ? host::launch(fl_rope_kernel<DT_F16, 8>, grid, kRopeThreads, 0, ctx.pdl, s, p)
                : host::launch(fl_rope_kernel<DT_F16, 1>, grid, kRopeThreads, 0, ctx.pdl, s, p);
    else
        e = vec ? host::launch(fl_rope_kernel<DT_BF16, 8>, grid, kRopeThreads, 0, ctx.pdl, s, p)
                : host::launch(fl_rope_kernel<DT_BF16, 1>, grid, kRopeThreads, 0, ctx.pdl, s, p);
    return host::launched(e, "rotary kernel");
}

}  // namespace

fl_status check_rope(const fl_rope_desc* desc) { return rope(desc, true, nullptr); }

}  // namespace fl

extern "C" fl_status fl_rope(const fl_rope_desc* desc, void* stream) {
    return fl::rope(desc, false, static_cast<cudaStream_t>(stream));
}
