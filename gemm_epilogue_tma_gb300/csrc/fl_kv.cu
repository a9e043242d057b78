// Paged 8-bit key/value cache: k and v rows quantised as they are written, and
// read back (fl_kv_write, fl_kv_read).
//
//   scale = max(amax * (1 / top), 2^-126), code = x / scale rounded to the format
//   x'    = scale * code
//
// with amax over the head_dim channels of one head's row and top = 127 (int8)
// or 448 (e4m3). Both kernels are bound by HBM: 3 bytes per channel (2 of the
// 16-bit side, 1 of the cache) and 4 per head's row.
//
// A lane takes 16 channels (8 where head_dim is not a multiple of 16), a head's
// row the smallest power-of-two group of lanes that holds it (8 lanes at
// head_dim 128), so amax is a butterfly over the group. One warp takes a row of
// both k and v, four passes of 32 lanes in flight, so that the look-up of the row's sequence
// and page, a chain of dependent loads, is made once for them; with few rows (a
// decode step) the passes are spread over more warps. The writing kernel
// requests its 16-bit vectors before the look-up.
//
// Measured in graphs: reading 60001 rows of 8 heads of 128 59 us (6.3 TB/s), writing
// 4099 9.4 us (2.7 TB/s, 25 MB: its inputs may be in L2; the codes' arithmetic
// and the launch are what is left; 8.7 us a call in an eager run); a decode step of 61
// sequences 2.7 us and 37 rows read 2.0 us, which is a launch and the look-up's
// loads one after another.
#include <cuda_fp8.h>

#include "fl_common.cuh"
#include "fl_host.h"
#include "fl_quant.cuh"

namespace fl {

namespace {

constexpr int kKvThreads = 128;
constexpr int kPasses = 4;       // passes of one reading warp task in flight
constexpr int kWritePasses = 2;  // and of a writing one, which also needs registers for its arithmetic (4: 10.8 against 9.4 us, 4099 rows)

struct KvParams {
    const uint16_t* src[2];  // write: k, v
    uint16_t* dst[2];        // read: k, v
    long long row[2], head[2];
    uint8_t* cache[2];
    float* scale[2];
    const int* page_table;
    const int* cu_rows;
    const int* start;
    long long table_stride;
    int rows, heads, head_dim, page_size, n_pages, n_seqs, table_pages;
    int lanes_log;  // lanes of one head's row: a power of two
    int half;       // passes of one row of k (or v)
    int per_task;   // passes of one warp task
    int tasks_row;  // warp tasks of one row
    uint32_t tasks;
    int* range;
};

// Place of row i in the cache (page * page_size + row in the page), -1 if it
// belongs to no sequence, -2 if its position has no page. Whole warp; every
// lane gets the answer. Among up to 128 sequences the one that holds the row is
// found in one step, in which each lane also loads what the answer will need of its
// sequences, so the look-up is two dependent loads, this one and the page;
// more sequences are narrowed down first, 32 offsets at a time.
__device__ __forceinline__ long long find_slot(const KvParams& p, int i, int lane) {
    int b, first = 0, from = 0;
    if (p.cu_rows == nullptr) {
        if (i >= p.n_seqs) return -1;
        b = first = i;
        if (p.start != nullptr) from = __ldg(p.start + b);
    } else {
        // the number of entries of cu_rows[1 ..] that are <= i
        constexpr int J = 4;       // sequences per lane in the last step
        int lo = 0, n = p.n_seqs;  // the answer is in [lo, lo + n]
        while (n > 32 * J) {
            const int step = (n + 31) / 32;
            const int at = min(lo + (lane + 1) * step, lo + n);  // candidates lo + step, lo + 2 step, .., lo + n
            const bool le = __ldg(p.cu_rows + at) <= i;
            const int c = __popc(__ballot_sync(0xffffffffu, le && lo + (lane + 1) * step <= lo + n + step - 1));
            // the first c candidates are <= i
            const int done = min(c * step, n);
            lo += done;
            n = done == n ? 0 : min(step - 1, n - done);
        }
        int end[J], begin[J], s[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int mine = min(lo + 32 * j + lane, p.n_seqs - 1);
            if (j == 0 || 32 * j < n) {
                end[j] = __ldg(p.cu_rows + mine + 1);
                begin[j] = __ldg(p.cu_rows + mine);
                s[j] = p.start != nullptr ? __ldg(p.start + mine) : 0;
            }
        }
        int c = 0;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (j == 0 || 32 * j < n) c += __popc(__ballot_sync(0xffffffffu, 32 * j + lane < n && end[j] <= i));
        b = lo + c;
        if (b >= p.n_seqs) return -1;
        int fb = begin[0], fs = s[0];
#pragma unroll
        for (int j = 1; j < J; ++j)
            if (c >= 32 * j && 32 * j < n) fb = begin[j], fs = s[j];
        if (c < 32 * ((max(n, 1) + 31) / 32)) {
            first = __shfl_sync(0xffffffffu, fb, c & 31);
            from = __shfl_sync(0xffffffffu, fs, c & 31);
        } else {
            first = __ldg(p.cu_rows + b);
            if (p.start != nullptr) from = __ldg(p.start + b);
        }
        if (i < first) return -1;
    }
    const long long pos = (long long)(i - first) + from;
    if (pos < 0 || pos >= (long long)p.table_pages * p.page_size) return -2;
    const uint32_t at = (uint32_t)pos, j = at / (uint32_t)p.page_size;  // (two int32 added: below 2^32)
    const int page = __ldg(p.page_table + b * p.table_stride + j);
    if (page < 0 || page >= p.n_pages) return -2;
    return (long long)page * p.page_size + (at - j * (uint32_t)p.page_size);
}

// What encoding a head's row needs of its scale s.
struct Quant {
    float up, dn;      // 1 / s, within 2^-23 of it, times 1 +- 2^-21
    float lift, half;  // s * lift / 2; lift is 2^64 for a tiny s, so that no residual underflows
    __device__ __forceinline__ explicit Quant(float s) {
        const float inv = rcp_approx(s);
        up = inv * (1.0f + 0x1p-21f), dn = inv * (1.0f - 0x1p-21f);
        lift = s < 0x1p-40f ? 0x1p64f : 1.0f;
        half = 0.5f * (s * lift);
    }
};

// Whether x / s rounds to `up` rather than to `dn`, the values of the two
// neighbouring codes it lies between (or of one code twice): the sign of
// x - (up + dn) / 2 * s, one FMA, says on which side of the border it is; on the
// border itself the even code is taken.
__device__ __forceinline__ bool takes_up(float x, float up, float dn, bool up_even, const Quant& q) {
    const float d = fmaf(-(up + dn), q.half, x * q.lift);
    return d == 0.f ? up_even : (d > 0.f) == (x > 0.f);
}

// Codes of 8 values. The quotient lies between x * dn and x * up, and rounding
// is monotonic, so where both round to the same code it is the exact
// quotient's. The others are decided exactly: far more than the width of the
// interval says (1 % of bf16 values), since 16-bit values are apt to lie on or
// next to a border (x = amax / 2 for int8).
//   int8: fma(x, up, 1.5 * 2^23) has the integer in its low bits.
template <int DT, int FMT>
__device__ __forceinline__ uint2 encode8(const uint4& v, const Quant& q) {
    using Ops = DTypeOps<DT>;
    constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = Ops::unpack(w[e]);
        if constexpr (FMT == FL_KV_INT8) {
            float a = fmaf(f.x, q.up, kShift), b = fmaf(f.y, q.up, kShift);
            const float a1 = fmaf(f.x, q.dn, kShift), b1 = fmaf(f.y, q.dn, kShift);
            if (a != a1 || b != b1) {
                if (!takes_up(f.x, a - kShift, a1 - kShift, (__float_as_uint(a) & 1u) == 0u, q)) a = a1;
                if (!takes_up(f.y, b - kShift, b1 - kShift, (__float_as_uint(b) & 1u) == 0u, q)) b = b1;
            }
            c[e] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
        } else {
            auto code = [](float a, float b) {
                return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
            };
            auto value = [](uint32_t k) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)k, __NV_E4M3);
                return __half22float2(*reinterpret_cast<const __half2*>(&h));
            };
            uint32_t k = code(f.x * q.up, f.y * q.up);
            const uint32_t k1 = code(f.x * q.dn, f.y * q.dn);
            if (k != k1) {
                const float2 a = value(k), a1 = value(k1);
                const bool x = takes_up(f.x, a.x, a1.x, (k & 1u) == 0u, q), y = takes_up(f.y, a.y, a1.y, (k & 0x100u) == 0u, q);
                k = ((x ? k : k1) & 0xffu) | ((y ? k : k1) & 0xff00u);
            }
            c[e] = k;
        }
    }
    return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

template <int DT, int FMT>
__device__ __forceinline__ uint4 decode8(uint2 c, float s) {
    using Ops = DTypeOps<DT>;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = e < 2 ? c.x : c.y;
        float2 f;
        if constexpr (FMT == FL_KV_INT8) {
            // the byte plus 128 in the mantissa of 2^23
            const uint32_t b = w ^ 0x80808080u;
            f.x = __uint_as_float(__byte_perm(b, 0x4b000000u, 0x7440 + 2 * (e & 1))) - 8388736.0f;
            f.y = __uint_as_float(__byte_perm(b, 0x4b000000u, 0x7441 + 2 * (e & 1))) - 8388736.0f;
        } else {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (e & 1))), __NV_E4M3);
            f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        }
        o[e] = Ops::pack(f.x * s, f.y * s);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A warp task: the passes [p0, p1) of row i; pass p is the p % half-th group of
// head rows of k (p < half) or v.
struct Task {
    int i, p0, p1;
};
__device__ __forceinline__ Task task_of(const KvParams& p, uint32_t t) {
    const uint32_t row = t / (uint32_t)p.tasks_row;
    const int p0 = (int)(t - row * (uint32_t)p.tasks_row) * p.per_task;
    return Task{(int)row, p0, min(p0 + p.per_task, 2 * p.half)};
}
// Where this lane's values of a pass are: pass q takes the head rows (q mod half)
// * groups + grp of k (q < half) or v.
template <int W, typename T>
struct Lane {
    T* x[2];            // its first pass's 16-bit values of k and v
    long long step[2];  // elements from one pass to the next
    int grp, sub, groups;
    bool in;
    __device__ __forceinline__ Lane(const KvParams& p, T* const (&base)[2], int row, int lane) {
        sub = lane & ((1 << p.lanes_log) - 1), grp = lane >> p.lanes_log, groups = 32 >> p.lanes_log;
        in = sub * (8 * W) < p.head_dim;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            x[w] = base[w] + row * p.row[w] + grp * p.head[w] + sub * (8 * W);
            step[w] = groups * p.head[w];
        }
    }
};

// W: 16-byte vectors of 16-bit values per lane (1 or 2).
template <int DT, int FMT, int W>
__global__ void __launch_bounds__(kKvThreads) fl_kv_write_kernel(const __grid_constant__ KvParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t t = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.tasks) return;
    const int lane = threadIdx.x & 31;
    const Task k = task_of(p, t);
    const Lane<W, const uint16_t> l(p, p.src, k.i, lane);
    long long slot = 0;
    for (int q0 = k.p0; q0 < k.p1; q0 += kWritePasses) {
        uint4 v[kWritePasses][W];
#pragma unroll
        for (int j = 0; j < kWritePasses; ++j) {
            const int q = q0 + j, w = q >= p.half, c = w ? q - p.half : q;
            const bool in = l.in && q < k.p1 && c * l.groups + l.grp < p.heads;
            const uint16_t* src = (w ? l.x[1] : l.x[0]) + c * (w ? l.step[1] : l.step[0]);
#pragma unroll
            for (int e = 0; e < W; ++e) v[j][e] = in ? ldg_v4(src + 8 * e) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (q0 == k.p0) {
            slot = find_slot(p, k.i, lane);
            if (slot < 0) {
                if (slot == -2 && lane == 0) atomicCAS(p.range, 0, k.i + 1);
                return;
            }
        }
#pragma unroll
        for (int j = 0; j < kWritePasses; ++j) {
            uint32_t m = absmax8<DT>(v[j][0]);
            if (W == 2) m = absmax2<DT>(m, absmax8<DT>(v[j][W - 1]));
            for (int o = 1 << p.lanes_log >> 1; o > 0; o >>= 1) m = absmax2<DT>(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int q = q0 + j, w = q >= p.half, h = (w ? q - p.half : q) * l.groups + l.grp;
            if (!l.in || q >= k.p1 || h >= p.heads) continue;
            m = absmax_halves<DT>(m);
            const bool fine = m < Bits16<DT>::kInf;
            const float s = fmaxf(DTypeOps<DT>::unpack(m).x * (1.0f / (FMT == FL_KV_INT8 ? 127.0f : 448.0f)), 0x1p-126f);
            const Quant quant(s);
            const long long at = slot * p.heads + h;
            if (l.sub == 0) p.scale[w][at] = fine ? s : __int_as_float(0x7fffffff);
            uint2 c[W];
#pragma unroll
            for (int e = 0; e < W; ++e) c[e] = fine ? encode8<DT, FMT>(v[j][e], quant) : make_uint2(0u, 0u);
            uint8_t* dst = p.cache[w] + at * p.head_dim + l.sub * (8 * W);
            if constexpr (W == 2)
                *reinterpret_cast<uint4*>(dst) = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
            else
                *reinterpret_cast<uint2*>(dst) = c[0];
        }
    }
}

template <int DT, int FMT, int W>
__global__ void __launch_bounds__(kKvThreads) fl_kv_read_kernel(const __grid_constant__ KvParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t t = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.tasks) return;
    const int lane = threadIdx.x & 31;
    const Task k = task_of(p, t);
    const long long slot = find_slot(p, k.i, lane);
    if (slot < 0) {
        if (slot == -2 && lane == 0) atomicCAS(p.range, 0, k.i + 1);
        return;
    }
    const Lane<W, uint16_t> l(p, p.dst, k.i, lane);
    for (int q0 = k.p0; q0 < k.p1; q0 += kPasses) {
        uint2 c[kPasses][W];
        float s[kPasses];
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
            // (a lane with nothing to read in this pass reads the place's first head row, so that all loads go out together)
            const int q = min(q0 + j, k.p1 - 1), w = q >= p.half, h = (w ? q - p.half : q) * l.groups + l.grp;
            const bool in = l.in && h < p.heads;
            const long long at = slot * p.heads + (in ? h : 0);
            const uint8_t* src = p.cache[w] + at * p.head_dim + (in ? l.sub * (8 * W) : 0);
            if constexpr (W == 2) {
                const uint4 x = ldg_v4(src);
                c[j][0] = make_uint2(x.x, x.y);
                c[j][W - 1] = make_uint2(x.z, x.w);
            } else {
                c[j][0] = __ldg(reinterpret_cast<const uint2*>(src));
            }
            s[j] = __ldg(p.scale[w] + at);
        }
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
            const int q = q0 + j, w = q >= p.half, i = w ? q - p.half : q;
            if (!l.in || q >= k.p1 || i * l.groups + l.grp >= p.heads) continue;
            uint16_t* dst = (w ? l.x[1] : l.x[0]) + i * (w ? l.step[1] : l.step[0]);
#pragma unroll
            for (int e = 0; e < W; ++e) *reinterpret_cast<uint4*>(dst + 8 * e) = decode8<DT, FMT>(c[j][e], s[j]);
        }
    }
}

fl_status check_desc(const char* what, const fl_kv_desc* d, bool write) {
    using host::fail;
    if (d == nullptr) return fail(FL_ERR_INVALID_ARG, "%s: null description", what);
    if (!host::valid_dtype(d->dtype)) return fail(FL_ERR_INVALID_ARG, "%s: bad dtype %d", what, (int)d->dtype);
    if (d->format != FL_KV_INT8 && d->format != FL_KV_E4M3)
        return fail(FL_ERR_INVALID_ARG, "%s: bad cache format %d", what, (int)d->format);
    if (d->rows < 0 || d->heads < 1 || d->head_dim < 1 || d->page_size < 1 || d->n_pages < 1 || d->n_seqs < 1 ||
        d->table_pages < 1)
        return fail(FL_ERR_INVALID_ARG, "%s: sizes must be positive (rows may be 0)", what);
    if (d->n_seqs > 1 << 30) return fail(FL_ERR_UNSUPPORTED, "%s: more than 2^30 sequences", what);
    if (d->head_dim % 8 != 0)
        return fail(FL_ERR_ALIGNMENT, "%s: head_dim must be a multiple of 8 (%d)", what, d->head_dim);
    if (d->head_dim > 256) return fail(FL_ERR_UNSUPPORTED, "%s: head_dim above 256 (%d)", what, d->head_dim);
    if (d->table_stride < 0 || (d->n_seqs > 1 && d->table_stride < d->table_pages))
        return fail(FL_ERR_INVALID_ARG, "%s: table_stride below table_pages", what);
    if (d->rows == 0) return FL_OK;
    fl_status st;
    if ((st = host::check_ptr("k", d->k, true)) != FL_OK) return st;
    if ((st = host::check_ptr("v", d->v, true)) != FL_OK) return st;
    if ((st = host::check_ptr("k_cache", d->k_cache, true)) != FL_OK) return st;
    if ((st = host::check_ptr("v_cache", d->v_cache, true)) != FL_OK) return st;
    if ((st = host::check_ptr("k_scale", d->k_scale, true)) != FL_OK) return st;
    if ((st = host::check_ptr("v_scale", d->v_scale, true)) != FL_OK) return st;
    if (d->page_table == nullptr) return fail(FL_ERR_INVALID_ARG, "page_table must not be null");
    const uintptr_t words = reinterpret_cast<uintptr_t>(d->page_table) | reinterpret_cast<uintptr_t>(d->cu_rows) |
                            reinterpret_cast<uintptr_t>(d->start);
    if (words & 3u) return fail(FL_ERR_ALIGNMENT, "page_table, cu_rows and start must be 4-byte aligned");
    // outputs: a row's heads lie inside its stride, or the rows inside a
    // head's, so that no two elements share a place
    const long long row[2] = {d->k_row, d->v_row}, head[2] = {d->k_head, d->v_head};
    for (int i = 0; i < 2; ++i) {
        if (row[i] % 8 != 0 || head[i] % 8 != 0)
            return fail(FL_ERR_ALIGNMENT, "%s: strides must be multiples of 8 elements", what);
        if (row[i] < 0 || head[i] < 0) return fail(FL_ERR_INVALID_ARG, "%s: negative stride", what);
        if (write) continue;
        if ((d->heads > 1 && head[i] < d->head_dim) || (d->rows > 1 && row[i] < d->head_dim))
            return fail(FL_ERR_INVALID_ARG, "%s: a stride below head_dim", what);
        const long long by_row = (d->heads - 1) * head[i] + d->head_dim, by_head = (d->rows - 1) * row[i] + d->head_dim;
        if (d->rows > 1 && d->heads > 1 && row[i] < by_row && head[i] < by_head)
            return fail(FL_ERR_INVALID_ARG, "%s: strides make rows overlap", what);
    }
    return FL_OK;
}

fl_status run(const char* what, const fl_kv_desc* d, bool write, bool check_only, cudaStream_t stream) {
    fl_status st = check_desc(what, d, write);
    if (st != FL_OK) return st;
    if (d->rows == 0) return host::ok();
    // outputs overlap neither one another nor an input
    const size_t places = (size_t)d->n_pages * d->page_size * d->heads;
    const size_t span[2] = {((size_t)(d->rows - 1) * d->k_row + (size_t)(d->heads - 1) * d->k_head + d->head_dim) * 2,
                            ((size_t)(d->rows - 1) * d->v_row + (size_t)(d->heads - 1) * d->v_head + d->head_dim) * 2};
    const size_t table = ((size_t)(d->n_seqs - 1) * d->table_stride + d->table_pages) * 4;
    struct Range {
        const void* p;
        size_t n;
        bool out;
    };
    const Range all[9] = {{d->k, span[0], !write},
                          {d->v, span[1], !write},
                          {d->k_cache, places * d->head_dim, write},
                          {d->v_cache, places * d->head_dim, write},
                          {d->k_scale, places * 4, write},
                          {d->v_scale, places * 4, write},
                          {d->page_table, table, false},
                          {d->cu_rows, (size_t)(d->n_seqs + 1) * 4, false},
                          {d->start, (size_t)d->n_seqs * 4, false}};
    for (int i = 0; i < 9; ++i)
        for (int j = 0; j < 9; ++j) {
            if (i == j || !all[i].out) continue;
            // k and v may be column ranges of one matrix, interleaved row by row
            if (i < 2 && j < 2 && host::apart(d->k, d->k_row, (d->heads - 1) * d->k_head + d->head_dim, d->v, d->v_row,
                                              (d->heads - 1) * d->v_head + d->head_dim, 2))
                continue;
            if (host::overlap(all[i].p, all[i].n, all[j].p, all[j].n))
                return host::fail(FL_ERR_INVALID_ARG, "%s: an output overlaps another tensor of the call", what);
        }
    const int W = d->head_dim % 16 == 0 ? 2 : 1;
    int lanes_log = 0;
    while ((8 * W << lanes_log) < d->head_dim) ++lanes_log;
    const int groups = 32 >> lanes_log, half = (d->heads + groups - 1) / groups;
    if (2ll * d->rows * half >= (1ll << 31)) return host::fail(FL_ERR_UNSUPPORTED, "%s: too many rows", what);
    if (check_only) return host::ok();
    host::LaunchContext ctx;
    if ((st = host::launch_context(stream, &ctx)) != FL_OK) return st;
    KvParams p = {};
    p.src[0] = p.dst[0] = static_cast<uint16_t*>(d->k);
    p.src[1] = p.dst[1] = static_cast<uint16_t*>(d->v);
    p.row[0] = d->k_row, p.row[1] = d->v_row, p.head[0] = d->k_head, p.head[1] = d->v_head;
    p.cache[0] = static_cast<uint8_t*>(d->k_cache), p.cache[1] = static_cast<uint8_t*>(d->v_cache);
    p.scale[0] = d->k_scale, p.scale[1] = d->v_scale;
    p.page_table = d->page_table, p.cu_rows = d->cu_rows, p.start = d->start;
    p.table_stride = d->table_stride;
    p.rows = d->rows, p.heads = d->heads, p.head_dim = d->head_dim, p.page_size = d->page_size;
    p.n_pages = d->n_pages, p.n_seqs = d->n_seqs, p.table_pages = d->table_pages;
    p.lanes_log = lanes_log, p.half = half;
    // a whole row to a warp once that gives every scheduler several warps
    p.per_task = 2 * half;
    while (p.per_task > 1 && (long long)d->rows * ((2 * half + p.per_task - 1) / p.per_task) < 16ll * ctx.sms)
        p.per_task = (p.per_task + 1) / 2;
    p.tasks_row = (2 * half + p.per_task - 1) / p.per_task;
    p.tasks = (uint32_t)d->rows * (uint32_t)p.tasks_row;
    p.range = ctx.range;
    const dim3 grid((p.tasks + kKvThreads / 32 - 1) / (kKvThreads / 32));
    cudaError_t e = cudaErrorInvalidValue;
#define FL_CASE(DT, FMT, WW)                                                                               \
    if (d->dtype == DT && d->format == FMT && W == WW)                                                     \
    e = write ? host::launch(fl_kv_write_kernel<DT, FMT, WW>, grid, kKvThreads, 0, ctx.pdl, stream, p)     \
              : host::launch(fl_kv_read_kernel<DT, FMT, WW>, grid, kKvThreads, 0, ctx.pdl, stream, p);
    FL_CASE(0, 0, 1) FL_CASE(0, 0, 2) FL_CASE(0, 1, 1) FL_CASE(0, 1, 2)
    FL_CASE(1, 0, 1) FL_CASE(1, 0, 2) FL_CASE(1, 1, 1) FL_CASE(1, 1, 2)
#undef FL_CASE
    return host::launched(e, what);
}

}  // namespace

fl_status check_kv_write(const fl_kv_desc* desc) { return run("fl_kv_write", desc, true, true, nullptr); }

}  // namespace fl

extern "C" fl_status fl_kv_write(const fl_kv_desc* desc, void* stream) {
    return fl::run("fl_kv_write", desc, true, false, static_cast<cudaStream_t>(stream));
}

extern "C" fl_status fl_kv_read(const fl_kv_desc* desc, void* stream) {
    return fl::run("fl_kv_read", desc, false, false, static_cast<cudaStream_t>(stream));
}
