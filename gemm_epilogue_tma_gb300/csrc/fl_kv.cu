// Paged 8-bit key/value cache: k and v rows quantised as they are written, and
// read back (fl_kv_write, fl_kv_read).
//
//   scale = max(amax / top, 2^-126), code = x / scale rounded to the format
//   x'    = scale * code
//
// with amax over the head_dim channels of one head's row and top = 127 (int8)
// or 448 (e4m3). Both kernels are bound by HBM: 3 bytes per channel (2 of the
// 16-bit side, 1 of the cache) and 4 per head's row.
//
// A head's row is handled by the smallest power-of-two group of lanes that
// holds it in 16-byte vectors (16 lanes at head_dim 128), so amax is a
// butterfly over the group. One warp takes a row of k or of v (or kVecs
// vectors per lane of it) at a time; its 16-bit vectors are requested before
// the row's sequence and page are looked up, so a decode step pays for the
// look-up's dependent loads and the data once, side by side.
#include <cuda_fp8.h>

#include "fl_common.cuh"
#include "fl_host.h"
#include "fl_quant.cuh"

namespace fl {

namespace {

constexpr int kKvThreads = 128;
constexpr int kVecs = 4;  // 16-byte vectors per lane in flight

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
    int lanes;   // lanes of one head's row (power of two)
    int chunks;  // warp tasks of one row of k (or v)
    int* range;
};

// Place of row i in the cache (page * page_size + row in the page), -1 if it
// belongs to no sequence, -2 if its position has no page. Whole warp; every
// lane gets the answer. The sequence is found 32 offsets at a time: first the
// block of a 32-ary split that holds it, then inside.
__device__ __forceinline__ long long find_slot(const KvParams& p, int i, int lane) {
    int b;
    long long pos;
    if (p.cu_rows == nullptr) {
        if (i >= p.n_seqs) return -1;
        b = i;
        pos = 0;
    } else {
        // the number of entries of cu_rows[1 ..] that are <= i
        int lo = 0, n = p.n_seqs;  // the answer is in [lo, lo + n]
        while (n > 0) {
            const int step = (n + 31) / 32;
            const int at = min(lo + (lane + 1) * step, lo + n);  // candidates lo + step, lo + 2 step, .., lo + n
            const bool le = __ldg(p.cu_rows + at) <= i;
            const int c = __popc(__ballot_sync(0xffffffffu, le && lo + (lane + 1) * step <= lo + n + step - 1));
            // the first c candidates are <= i
            const int done = min(c * step, n);
            lo += done;
            n = done == n ? 0 : min(step - 1, n - done);
        }
        if (lo >= p.n_seqs) return -1;
        b = lo;
        const int first = __ldg(p.cu_rows + b);
        if (i < first) return -1;
        pos = i - first;
    }
    if (p.start != nullptr) pos += __ldg(p.start + b);
    if (pos < 0 || pos >= (long long)p.table_pages * p.page_size) return -2;
    const uint32_t at = (uint32_t)pos, j = at / (uint32_t)p.page_size;  // (two int32 added: below 2^32)
    const int page = __ldg(p.page_table + b * p.table_stride + j);
    if (page < 0 || page >= p.n_pages) return -2;
    return (long long)page * p.page_size + (at - j * (uint32_t)p.page_size);
}

// int8 code of x: round(x / s) with inv = 1 / s rounded. x * inv is within two
// units in the last place of the quotient, so only a quotient next to a border
// between two codes can round to the wrong side: there the sign of
// x - (border) * s, one FMA, decides, and 0 is a tie, which goes to even.
__device__ __forceinline__ int code_int8(float x, float s, float inv) {
    const float y = x * inv;
    float r = rintf(y);
    if (fabsf(y - r) > 0.4999f) {
        const float lo = floorf(y), d = fmaf(-(lo + 0.5f), s, x);
        r = d > 0.f ? lo + 1.f : d < 0.f ? lo : 2.f * rintf(0.5f * (lo + 0.5f));
    }
    return (int)fminf(fmaxf(r, -127.f), 127.f);
}

// x / s with its last bit set when the quotient is not exact (rounding to
// odd), so that the conversion to e4m3, which keeps 4 of the 24 bits, rounds
// the exact quotient: x * inv, one Newton step, then the residual's sign.
__device__ __forceinline__ float odd_quotient(float x, float s, float inv) {
    float y = x * inv;
    y = fmaf(fmaf(-y, s, x), inv, y);
    const float e = fmaf(-y, s, x);
    uint32_t u = __float_as_uint(y);
    if (e != 0.f && (u & 1u) == 0u && (u << 1) != 0u) u += ((__float_as_uint(e) ^ u) >> 31) ? 0xffffffffu : 1u;
    return __uint_as_float(u);
}

template <int DT, int FMT>
__device__ __forceinline__ uint2 encode8(const uint4& v, float s) {
    using Ops = DTypeOps<DT>;
    const float inv = 1.0f / s;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = Ops::unpack(w[e]);
        if constexpr (FMT == FL_KV_INT8) {
            const int a = code_int8(f.x, s, inv), b = code_int8(f.y, s, inv);
            o[e] = (a & 0xff) | ((b & 0xff) << 8);
        } else {
            o[e] = __nv_cvt_float2_to_fp8x2(make_float2(odd_quotient(f.x, s, inv), odd_quotient(f.y, s, inv)),
                                            __NV_SATFINITE, __NV_E4M3);
        }
    }
    return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

template <int DT, int FMT>
__device__ __forceinline__ uint4 decode8(uint2 c, float s) {
    using Ops = DTypeOps<DT>;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = ((e < 2 ? c.x : c.y) >> (16 * (e & 1))) & 0xffffu;
        float2 f;
        if constexpr (FMT == FL_KV_INT8) {
            f = make_float2((float)(int8_t)(w & 0xff), (float)(int8_t)(w >> 8));
        } else {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
            f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        }
        o[e] = Ops::pack(f.x * s, f.y * s);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// One warp task: row i of k (which = 0) or v, head rows [h0, h0 + units).
struct Task {
    int i, which, h0, units;
};
__device__ __forceinline__ Task task_of(const KvParams& p, uint32_t t) {
    const int per = 32 / p.lanes * kVecs;
    Task k;
    const uint32_t rest = t / (uint32_t)p.chunks;
    k.which = (int)(rest & 1u);
    k.i = (int)(rest >> 1);
    k.h0 = (int)(t - rest * (uint32_t)p.chunks) * per;
    k.units = min(per, p.heads - k.h0);
    return k;
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kKvThreads) fl_kv_write_kernel(const __grid_constant__ KvParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane & (p.lanes - 1), grp = lane / p.lanes, groups = 32 / p.lanes;
    const uint32_t tasks = 2u * p.rows * p.chunks, stride = gridDim.x * (kKvThreads / 32);
    for (uint32_t t = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5); t < tasks; t += stride) {
        const Task k = task_of(p, t);
        const bool in = sub * 8 < p.head_dim;
        const uint16_t* src = p.src[k.which] + k.i * p.row[k.which] + sub * 8;
        uint4 v[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int h = u * groups + grp;
            v[u] = in && h < k.units ? ldg_v4(src + (k.h0 + h) * p.head[k.which]) : make_uint4(0u, 0u, 0u, 0u);
        }
        const long long slot = find_slot(p, k.i, lane);
        if (slot < 0) {
            if (slot == -2 && lane == 0) atomicCAS(p.range, 0, k.i + 1);
            continue;
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int h = u * groups + grp;
            uint32_t m = absmax8<DT>(v[u]);
            for (int o = p.lanes / 2; o > 0; o >>= 1) m = absmax2<DT>(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (h >= k.units) continue;
            const bool fine = (m & 0xffffu) < Bits16<DT>::kInf;
            const float top = FMT == FL_KV_INT8 ? 127.0f : 448.0f;
            const float s = fmaxf(DTypeOps<DT>::unpack(m).x / top, 0x1p-126f);
            const long long at = slot * p.heads + k.h0 + h;
            if (sub == 0) p.scale[k.which][at] = fine ? s : __int_as_float(0x7fffffff);
            if (in)
                *reinterpret_cast<uint2*>(p.cache[k.which] + at * p.head_dim + sub * 8) =
                    fine ? encode8<DT, FMT>(v[u], s) : make_uint2(0u, 0u);
        }
    }
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kKvThreads) fl_kv_read_kernel(const __grid_constant__ KvParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane & (p.lanes - 1), grp = lane / p.lanes, groups = 32 / p.lanes;
    const uint32_t tasks = 2u * p.rows * p.chunks, stride = gridDim.x * (kKvThreads / 32);
    for (uint32_t t = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5); t < tasks; t += stride) {
        const Task k = task_of(p, t);
        const long long slot = find_slot(p, k.i, lane);
        if (slot < 0) {
            if (slot == -2 && lane == 0) atomicCAS(p.range, 0, k.i + 1);
            continue;
        }
        const bool in = sub * 8 < p.head_dim;
        uint2 c[kVecs];
        float s[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int h = u * groups + grp;
            if (!in || h >= k.units) continue;
            const long long at = slot * p.heads + k.h0 + h;
            c[u] = __ldg(reinterpret_cast<const uint2*>(p.cache[k.which] + at * p.head_dim + sub * 8));
            s[u] = __ldg(p.scale[k.which] + at);
        }
        uint16_t* dst = p.dst[k.which] + k.i * p.row[k.which] + sub * 8;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int h = u * groups + grp;
            if (!in || h >= k.units) continue;
            *reinterpret_cast<uint4*>(dst + (k.h0 + h) * p.head[k.which]) = decode8<DT, FMT>(c[u], s[u]);
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

fl_status run(const char* what, const fl_kv_desc* d, bool write, cudaStream_t stream) {
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
    int lanes = 1;
    while (lanes * 8 < d->head_dim) lanes *= 2;
    const int per = 32 / lanes * kVecs, chunks = (d->heads + per - 1) / per;
    if (2ll * d->rows * chunks >= (1ll << 31)) return host::fail(FL_ERR_UNSUPPORTED, "%s: too many rows", what);
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
    p.lanes = lanes, p.chunks = chunks;
    p.range = ctx.range;
    const long long ctas = (2ll * d->rows * p.chunks + kKvThreads / 32 - 1) / (kKvThreads / 32);
    const long long most = 16ll * ctx.sms;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    cudaError_t e;
#define FL_CASE(DT, FMT)                                                                                   \
    if (d->dtype == DT && d->format == FMT)                                                                \
        e = write ? host::launch(fl_kv_write_kernel<DT, FMT>, grid, kKvThreads, 0, ctx.pdl, stream, p)      \
                  : host::launch(fl_kv_read_kernel<DT, FMT>, grid, kKvThreads, 0, ctx.pdl, stream, p)
    e = cudaErrorInvalidValue;
    FL_CASE(0, 0);
    FL_CASE(0, 1);
    FL_CASE(1, 0);
    FL_CASE(1, 1);
#undef FL_CASE
    return host::launched(e, what);
}

}  // namespace

}  // namespace fl

extern "C" fl_status fl_kv_write(const fl_kv_desc* desc, void* stream) {
    return fl::run("fl_kv_write", desc, true, static_cast<cudaStream_t>(stream));
}

extern "C" fl_status fl_kv_read(const fl_kv_desc* desc, void* stream) {
    return fl::run("fl_kv_read", desc, false, static_cast<cudaStream_t>(stream));
}
