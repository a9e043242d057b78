// The pages of the paged cache: page tables brought to new lengths
// (fl_kv_resize), sequences that share another's pages (fl_kv_fork), and the rows
// of accepted drafts moved to the end of their contexts (fl_kv_compact).
//
// A page is free when no table entry holds it: refs[page] counts the entries.
// Tables and counts live on the GPU, so that a step that grows, verifies, keeps and
// cuts back can be captured into one graph. Pages are given out in ascending
// order to the entries that want one in ascending order (sequence, then place in
// its table): the answer depends on the arguments alone.
//
// Resize and fork are one kernel of one CTA for small tables, where a barrier costs
// little, or of one cluster of eight or sixteen. Each warp takes a run of
// neighbouring table segments of 256 entries and a run of neighbouring pages:
//   1. entries past the new length are released (refs - 1), wanting ones counted
//   2. free pages counted; both counts go to every CTA through distributed
//      shared memory, so that each warp knows how many stand in front of its own
//   3. the k-th free page is written to place k of a list, k below the wanted number
//   4. the k-th wanting entry takes page k of the list
// (a fork releases what its children held in a phase of its own, in front, and marks the entries that want a page)
// with a barrier after each. Nothing but latency bounds it: the barriers, and the rounds of
// loads of a warp's run, eight loads to a round. Graph times: two calls for seven sequences
// of 16 entries 6.9 us, for 256 of 1024 entries and 121000 pages 21; a fork of one
// sequence into three 8.0 with its copy, of eight into 56 11.9; rows of one tree moved 2.9, of 61 3.8.
#include <algorithm>

#include "fl_common.cuh"
#include "fl_host.h"

namespace fl {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 256;  // table entries of a warp at a time
constexpr int kPer = kSegment / 32;
constexpr int kWants = -2;     // fork: an entry that wants a page, between the phases (none, like every negative one)

struct PagesParams {
    int* page_table;
    int* refs;
    const int* lengths;
    const int* parents;   // fork
    const int* children;
    int* list;            // free pages, at most n_pages
    long long table_stride;
    int n, n_seqs, table_pages, n_pages, page_size;  // n: sequences (resize) or children (fork)
    int* range;
};

// Sum over the cluster's warps in front of this one, and over all of them, of a
// count per warp. Whole cluster, one barrier; `slot` is this phase's shared memory.
struct Share {
    int mine[kWarps];
    int total;
};
__device__ __forceinline__ void publish(Share& s, int count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s.mine[warp] = count;
    __syncthreads();
    if (warp == 0) {
        int v = s.mine[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s.total = v;
    }
}
template <int CTAS>
__device__ __forceinline__ void all_sync() {
    if constexpr (CTAS == 1) __syncthreads();
    else cluster_barrier_sync();
}
template <int CTAS>
__device__ __forceinline__ void collect(Share& s, int& before, int& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 1 ? 0u : cluster_rank();
    int v = 0, w = lane < warp ? s.mine[lane] : 0;
    if constexpr (CTAS == 1) {
        if (lane == 0) v = s.total;
    } else if (lane < CTAS)
        asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(mapa_cluster(smem_u32(&s.total), lane)) : "memory");
    if (CTAS > 1 && (uint32_t)lane < rank) w += v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v += __shfl_xor_sync(0xffffffffu, v, o);
        w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    before = w, all = v;
}

template <bool FORK, int CTAS>
__global__ void __launch_bounds__(kThreads, 1) fl_kv_pages_kernel(const __grid_constant__ PagesParams p) {
    __shared__ Share wanting, freed;
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int me = (CTAS == 1 ? 0 : (int)cluster_rank()) * kWarps + warp;
    constexpr int kAll = CTAS * kWarps;
    const int per_row = (p.table_pages + kSegment - 1) / kSegment;
    const long long segments = (long long)p.n * per_row;
    const long long s0 = segments * me / kAll, s1 = segments * (me + 1) / kAll;
    auto held = [&](int e) { return e >= 0 && e < p.n_pages; };
    auto valid = [&](int b) { return b >= 0 && b < p.n_seqs; };
    // whole pages and the rest of a length, within the table
    auto pages_of = [&](int len, int& part) {
        const int full = max(len, 0) / p.page_size;
        part = max(len, 0) - full * p.page_size;
        if (full >= p.table_pages) {
            if (full > p.table_pages || part > 0) atomicCAS(p.range, 0, 1);
            part = 0;
            return p.table_pages;
        }
        return full;
    };

    if (FORK) {
        // What the children held goes. (Exchanged, so that it goes once where a sequence is a child twice: that has no defined answer,
        // but no page of another sequence may become free.)
        for (long long s = s0; s < s1; ++s) {
            const int i = (int)(s / per_row), j0 = (int)(s % per_row) * kSegment;
            const int c = __ldg(p.children + i);
            if (!valid(c) || !valid(__ldg(p.parents + i))) continue;
            int* row = p.page_table + c * p.table_stride;
            int e[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int j = j0 + 32 * u + lane;
                e[u] = j < p.table_pages ? atomicExch(row + j, -1) : -1;
            }
#pragma unroll
            for (int u = 0; u < kPer; ++u)
                if (held(e[u])) atomicAdd(p.refs + e[u], -1);
        }
        all_sync<CTAS>();
    }
    // Entries of this warp's segments: want(u, j) for those that want a page.
    // Phase 0 releases or shares and counts, phase 1 gives pages.
    int count = 0;
    uint32_t wants_of = 0;  // resize: which of a lane's entries want a page, of the first 32 / kPer segments
    for (long long s = s0; s < s1; ++s) {
        const int i = (int)(s / per_row), j0 = (int)(s % per_row) * kSegment;
        int part;
        if (!FORK) {
            int* row = p.page_table + i * p.table_stride;
            int need = pages_of(__ldg(p.lengths + i), part);
            need += part > 0;
            int e[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int j = j0 + 32 * u + lane;
                e[u] = j < p.table_pages ? __ldcg(row + j) : -1;
            }
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int j = j0 + 32 * u + lane;
                if (j >= need && held(e[u])) {
                    atomicAdd(p.refs + e[u], -1);
                    row[j] = -1;
                }
                const bool wants = j < need && !held(e[u]);
                count += wants;
                if (s - s0 < 32 / kPer) wants_of |= (uint32_t)wants << ((int)(s - s0) * kPer + u);
            }
        } else {
            const int c = __ldg(p.children + i), from = __ldg(p.parents + i);
            if (!valid(c) || !valid(from)) {
                if (j0 == 0 && lane == 0) atomicCAS(p.range, 0, i + 1);
                continue;
            }
            int* row = p.page_table + c * p.table_stride;
            const int* parent = p.page_table + from * p.table_stride;
            const int full = pages_of(__ldg(p.lengths + i), part);
            int e[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int j = j0 + 32 * u + lane;
                e[u] = j < full + (part > 0) ? __ldcg(parent + j) : -1;
            }
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int j = j0 + 32 * u + lane;
                if (j >= p.table_pages) continue;
                const bool share = j < full && held(e[u]);
                if (share) atomicAdd(p.refs + e[u], 1);
                if (j < full + (part > 0) && !held(e[u])) atomicCAS(p.range, 0, i + 1);
                const bool wants = j == full && part > 0 && held(e[u]);
                row[j] = share ? e[u] : wants ? kWants : -1;
                count += wants;
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
    publish(wanting, count);
    all_sync<CTAS>();
    int rank, wanted, at, available;
    collect<CTAS>(wanting, rank, wanted);

    const int f0 = (int)((long long)p.n_pages * me / kAll), f1 = (int)((long long)p.n_pages * (me + 1) / kAll);
    if (wanted > 0) {  // (the same in the whole cluster)
        // (which of its pages are free: 32 rounds of a page to a lane are kept, more are read again)
        uint32_t flags = 0;
        auto free_at = [&](int q) { return q < f1 && __ldcg(p.refs + q) == 0; };
        count = 0;
        for (int i0 = 0; f0 + 32 * i0 < f1; i0 += kPer) {
            bool is[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) is[u] = free_at(f0 + 32 * (i0 + u) + lane);
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                count += is[u];
                if (i0 + u < 32) flags |= (uint32_t)is[u] << ((i0 + u) & 31);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
        publish(freed, count);
        all_sync<CTAS>();
        collect<CTAS>(freed, at, available);
        for (int i = 0; f0 + 32 * i < f1 && at < wanted; ++i) {
            const int q = f0 + 32 * i + lane;
            const bool is = i < 32 ? flags >> i & 1 : free_at(q);
            const uint32_t m = __ballot_sync(0xffffffffu, is);
            const int k = at + __popc(m & ((1u << lane) - 1));
            if (is && k < wanted) {
                p.list[k] = q;
                p.refs[q] = 1;
            }
            at += __popc(m);
        }
        all_sync<CTAS>();
        for (long long s = s0; s < s1; ++s) {
            const int i = (int)(s / per_row), j0 = (int)(s % per_row) * kSegment;
            int part = 0, limit, c = i;
            if (FORK) {
                c = __ldg(p.children + i);
                if (!valid(c) || !valid(__ldg(p.parents + i))) continue;
            }
            limit = pages_of(__ldg(p.lengths + i), part);
            const int first = FORK ? limit : 0;
            if (FORK && part == 0) continue;
            limit += part > 0;
            int* row = p.page_table + c * p.table_stride;
            // (all places in the list first, then all loads from it)
            int k[kPer], page[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int j = j0 + 32 * u + lane;
                bool wants = j >= first && j < limit && j < p.table_pages;
                if (FORK) wants = wants && __ldcg(row + j) == kWants;
                else wants = s - s0 < 32 / kPer ? wants_of >> ((int)(s - s0) * kPer + u) & 1 : wants && !held(__ldcg(row + j));
                const uint32_t m = __ballot_sync(0xffffffffu, wants);
                k[u] = wants ? rank + __popc(m & ((1u << lane) - 1)) : -1;
                rank += __popc(m);
            }
#pragma unroll
            for (int u = 0; u < kPer; ++u) page[u] = k[u] >= 0 && k[u] < available ? __ldcg(p.list + k[u]) : -1;
#pragma unroll
            for (int u = 0; u < kPer; ++u)
                if (k[u] >= 0) {
                    row[j0 + 32 * u + lane] = page[u];
                    if (k[u] >= available) atomicCAS(p.range, 0, i + 1);
                }
        }
    }
    // (the counts of this CTA may still be read by another; with pages given out there was a barrier since)
    if (CTAS > 1 && wanted == 0) all_sync<CTAS>();
}

// The rows of a parent's last, partly filled page into the child's: one
// (child, slice) to a CTA. k and v rows of a page are contiguous.
struct CopyParams {
    uint8_t* cache[2];
    float* scale[2];
    const int* page_table;
    const int* refs;
    const int* lengths;
    const int* parents;
    const int* children;
    long long table_stride, row_bytes;  // of one position's heads
    int heads, n_seqs, table_pages, n_pages, page_size;
};
constexpr int kCopyThreads = 256;
constexpr int kSlices = 8;

template <typename T, int U>
__device__ __forceinline__ void copy_run(T* dst, const T* src, long long n, int tid, int threads, bool own) {
    for (long long b = tid; b < n; b += (long long)threads * U) {
        T v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u * threads < n) v[u] = __ldcg(src + b + u * threads);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (own && b + u * threads < n) dst[b + u * threads] = v[u];
    }
}

__global__ void __launch_bounds__(kCopyThreads) fl_kv_fork_copy_kernel(const __grid_constant__ CopyParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int i = blockIdx.x, c = __ldg(p.children + i), from = __ldg(p.parents + i), len = __ldg(p.lengths + i);
    if (c < 0 || c >= p.n_seqs || from < 0 || from >= p.n_seqs || len <= 0) return;
    const int full = len / p.page_size, part = len - full * p.page_size;
    if (part == 0 || full >= p.table_pages) return;
    const int a = __ldcg(p.page_table + from * p.table_stride + full), b = __ldcg(p.page_table + c * p.table_stride + full);
    if (a < 0 || a >= p.n_pages || b < 0 || b >= p.n_pages || a == b) return;
    // The child's own page is held once; another than that stands here only where a sequence is a child twice. (Asked for beside the
    // rows, which are not stored otherwise.)
    const bool own = __ldcg(p.refs + b) == 1;
    const long long src = (long long)a * p.page_size, dst = (long long)b * p.page_size;
    const int tid = blockIdx.y * kCopyThreads + threadIdx.x, threads = kSlices * kCopyThreads;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint8_t* to = p.cache[w] + dst * p.row_bytes;
        const uint8_t* at = p.cache[w] + src * p.row_bytes;
        if (p.row_bytes % 16 == 0)
            copy_run<uint4, 4>(reinterpret_cast<uint4*>(to), reinterpret_cast<const uint4*>(at), part * p.row_bytes / 16, tid, threads, own);
        else
            copy_run<uint2, 4>(reinterpret_cast<uint2*>(to), reinterpret_cast<const uint2*>(at), part * p.row_bytes / 8, tid, threads, own);
        copy_run<float, 2>(p.scale[w] + dst * p.heads, p.scale[w] + src * p.heads, (long long)part * p.heads, tid, threads, own);
    }
}

// Rows start + accepted[j] -> start + j. A thread moves the same bytes of every
// row of its sequence, eight rows loaded before the first is stored: a row's
// source lies behind or at its place, and the sources ascend, so no
// row is read after it was overwritten, and no thread waits for another.
struct CompactParams {
    uint8_t* cache[2];
    float* scale[2];
    const int* page_table;
    const int* start;
    const int* accepted;  // [n_seqs][most]
    long long table_stride, row_bytes;
    int heads, most, table_pages, n_pages, page_size;
    int* range;
};
constexpr int kMoveThreads = 256;
constexpr int kChunk = 64;  // rows whose places are looked up at a time

template <typename T>
__device__ __forceinline__ void move_rows(T* base, long long pitch, const long long* src, const long long* dst, int n) {
    for (int j = 0; j < n; j += 8) {
        T v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (j + u < n && src[j + u] >= 0) v[u] = __ldcg(base + src[j + u] * pitch);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (j + u < n && src[j + u] >= 0) base[dst[j + u] * pitch] = v[u];
    }
}

template <typename T>
__global__ void __launch_bounds__(kMoveThreads) fl_kv_compact_kernel(const __grid_constant__ CompactParams p) {
    __shared__ long long src[kChunk], dst[kChunk];
    __shared__ int stop;
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x;
    const long long from = __ldg(p.start + b);
    const int* table = p.page_table + b * p.table_stride;
    const int* acc = p.accepted + (long long)b * p.most;
    const int words = (int)(p.row_bytes / (int)sizeof(T));
    const int col = blockIdx.y * kMoveThreads + threadIdx.x;
    auto place = [&](long long pos) -> long long {
        if (pos < 0 || pos >= (long long)p.table_pages * p.page_size) return -1;
        const uint32_t j = (uint32_t)pos / (uint32_t)p.page_size;
        const int page = __ldg(table + j);
        if (page < 0 || page >= p.n_pages) return -1;
        return (long long)page * p.page_size + (uint32_t)pos % (uint32_t)p.page_size;
    };
    for (int j0 = 0; j0 < p.most; j0 += kChunk) {
        if (threadIdx.x == 0) stop = min(kChunk, p.most - j0);
        __syncthreads();
        if (threadIdx.x < kChunk && j0 + (int)threadIdx.x < p.most) {
            const int j = j0 + threadIdx.x, a = __ldg(acc + j);
            src[threadIdx.x] = dst[threadIdx.x] = -1;
            if (a < 0) {
                atomicMin(&stop, (int)threadIdx.x);
            } else if (a != j) {
                const long long x = place(from + a), y = place(from + j);
                if (x >= 0 && y >= 0) {
                    src[threadIdx.x] = x, dst[threadIdx.x] = y;
                } else {
                    src[threadIdx.x] = -2;
                }
            }
        }
        __syncthreads();
        const int n = stop;
        // (reported for rows in front of the end alone)
        if (threadIdx.x < n && src[threadIdx.x] == -2) atomicCAS(p.range, 0, b + 1);
        if (col < 2 * words) {
            const int w = col >= words;
            move_rows(reinterpret_cast<T*>(p.cache[w]) + (col - w * words), words, src, dst, n);
        } else if (col < 2 * words + 2 * p.heads) {
            const int h = col - 2 * words, w = h >= p.heads;
            move_rows(p.scale[w] + (h - w * p.heads), p.heads, src, dst, n);
        }
        if (n < kChunk) return;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using host::fail;

struct Range {
    const void* p;
    size_t n;
    bool out;
};
template <int N>
fl_status check_ranges(const char* what, const Range (&all)[N]) {
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && all[i].out && (!all[j].out || i < j) && all[i].p != nullptr && all[j].p != nullptr &&
                host::overlap(all[i].p, all[i].n, all[j].p, all[j].n))
                return fail(FL_ERR_INVALID_ARG, "%s: a tensor that is written overlaps another of the call", what);
    return FL_OK;
}

fl_status check_ints(const char* what, const void* p) {
    if (p == nullptr) return fail(FL_ERR_INVALID_ARG, "%s: a required pointer is null", what);
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(FL_ERR_ALIGNMENT, "%s: pointers must be 4-byte aligned", what);
    return FL_OK;
}

fl_status check_table(const char* what, const fl_kv_pages* c) {
    if (c == nullptr) return fail(FL_ERR_INVALID_ARG, "%s: null cache", what);
    if (c->page_size < 1 || c->n_pages < 1 || c->n_seqs < 1 || c->table_pages < 1)
        return fail(FL_ERR_INVALID_ARG, "%s: sizes must be positive", what);
    if (c->n_seqs > 1 << 30) return fail(FL_ERR_UNSUPPORTED, "%s: more than 2^30 sequences", what);
    if (c->table_stride < 0 || (c->n_seqs > 1 && c->table_stride < c->table_pages))
        return fail(FL_ERR_INVALID_ARG, "%s: table_stride below table_pages", what);
    return check_ints(what, c->page_table);
}
size_t table_bytes(const fl_kv_pages* c) { return ((size_t)(c->n_seqs - 1) * c->table_stride + c->table_pages) * 4; }

fl_status check_cache(const char* what, const fl_kv_pages* c) {
    if (c->heads < 1 || c->head_dim < 1) return fail(FL_ERR_INVALID_ARG, "%s: sizes must be positive", what);
    if (c->head_dim % 8 != 0) return fail(FL_ERR_ALIGNMENT, "%s: head_dim must be a multiple of 8 (%d)", what, c->head_dim);
    if (c->head_dim > 256) return fail(FL_ERR_UNSUPPORTED, "%s: head_dim above 256 (%d)", what, c->head_dim);
    if (c->heads > 1 << 20) return fail(FL_ERR_UNSUPPORTED, "%s: more than 2^20 heads", what);
    fl_status st;
    if ((st = host::check_ptr("k_cache", c->k_cache, true)) != FL_OK) return st;
    if ((st = host::check_ptr("v_cache", c->v_cache, true)) != FL_OK) return st;
    if ((st = host::check_ptr("k_scale", c->k_scale, true)) != FL_OK) return st;
    return host::check_ptr("v_scale", c->v_scale, true);
}

template <bool FORK>
fl_status launch_pages(const char* what, const PagesParams& p, const host::LaunchContext& ctx, cudaStream_t stream) {
    // A segment to a warp decides: one CTA, eight or sixteen. Two resize calls, us, with 1 / 8 / 16 CTAs: seven
    // sequences of 16 entries and 79 pages 6.9 / 9.1 / 13.3; 61 of 256 and 10863 pages 14.0 / 11.1 / 14.2; 256 of
    // 1024 and 121048 pages 178 / 26.1 / 20.9; a fork of 8 to 56 children 15.6 / 11.9 / 15.2.
    const long long segments = (long long)p.n * ((p.table_pages + kSegment - 1) / kSegment);
    if (segments <= 32 && p.n_pages <= 2048)
        return host::launched(host::launch(fl_kv_pages_kernel<FORK, 1>, dim3(1), kThreads, 0, ctx.pdl, stream, p), what);
    if (segments <= 512 && p.n_pages <= 65536)
        return host::launched(host::launch_cluster(fl_kv_pages_kernel<FORK, 8>, dim3(8), kThreads, 0, ctx.pdl, 8, stream, p), what);
    static std::atomic<unsigned long long> done{0};
    if (!(done.load(std::memory_order_relaxed) >> ctx.device & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(fl_kv_pages_kernel<FORK, 16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return fail(FL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
        done.fetch_or(1ull << ctx.device, std::memory_order_relaxed);
    }
    return host::launched(host::launch_cluster(fl_kv_pages_kernel<FORK, 16>, dim3(16), kThreads, 0, ctx.pdl, 16, stream, p), what);
}

PagesParams pages_params(const fl_kv_pages* c, int* refs, const int* lengths, void* workspace, int* range) {
    PagesParams p = {};
    p.page_table = c->page_table, p.refs = refs, p.lengths = lengths, p.list = static_cast<int*>(workspace);
    p.table_stride = c->table_stride, p.n = p.n_seqs = c->n_seqs, p.table_pages = c->table_pages;
    p.n_pages = c->n_pages, p.page_size = c->page_size, p.range = range;
    return p;
}

fl_status check_workspace(const char* what, const fl_kv_pages* c, const void* workspace, size_t bytes) {
    const fl_status st = host::check_ptr("workspace", workspace, false);
    if (st != FL_OK) return st;
    const size_t need = fl_kv_pages_workspace_size(c->n_pages);
    if (workspace == nullptr || bytes < need)
        return fail(FL_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", what, need, bytes);
    return FL_OK;
}

}  // namespace

}  // namespace fl

extern "C" size_t fl_kv_pages_workspace_size(int n_pages) { return n_pages < 1 ? 0 : (size_t)n_pages * 4; }

extern "C" fl_status fl_kv_resize(const fl_kv_pages* cache, int* refs, const int* lengths, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    using namespace fl;
    const char* what = "fl_kv_resize";
    fl_status st;
    if ((st = check_table(what, cache)) != FL_OK) return st;
    if ((st = check_ints(what, refs)) != FL_OK) return st;
    if ((st = check_ints(what, lengths)) != FL_OK) return st;
    if ((st = check_workspace(what, cache, workspace, workspace_bytes)) != FL_OK) return st;
    const Range all[] = {{cache->page_table, table_bytes(cache), true},
                         {refs, (size_t)cache->n_pages * 4, true},
                         {workspace, (size_t)cache->n_pages * 4, true},
                         {lengths, (size_t)cache->n_seqs * 4, false}};
    if ((st = check_ranges(what, all)) != FL_OK) return st;
    host::LaunchContext ctx;
    if ((st = host::launch_context(static_cast<cudaStream_t>(stream), &ctx)) != FL_OK) return st;
    return launch_pages<false>(what, pages_params(cache, refs, lengths, workspace, ctx.range), ctx,
                               static_cast<cudaStream_t>(stream));
}

extern "C" fl_status fl_kv_fork(const fl_kv_pages* cache, int* refs, const int* parents, const int* children,
                                const int* lengths, int n, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace fl;
    const char* what = "fl_kv_fork";
    fl_status st;
    if ((st = check_table(what, cache)) != FL_OK) return st;
    if ((st = check_cache(what, cache)) != FL_OK) return st;
    if (n < 0) return fail(FL_ERR_INVALID_ARG, "%s: n must not be negative", what);
    if (n == 0) return host::ok();
    const void* ints[] = {refs, parents, children, lengths};
    for (const void* p : ints)
        if ((st = check_ints(what, p)) != FL_OK) return st;
    if ((st = check_workspace(what, cache, workspace, workspace_bytes)) != FL_OK) return st;
    const size_t places = (size_t)cache->n_pages * cache->page_size * cache->heads;
    const Range all[] = {{cache->page_table, table_bytes(cache), true},
                         {refs, (size_t)cache->n_pages * 4, true},
                         {workspace, (size_t)cache->n_pages * 4, true},
                         {cache->k_cache, places * cache->head_dim, true},
                         {cache->v_cache, places * cache->head_dim, true},
                         {cache->k_scale, places * 4, true},
                         {cache->v_scale, places * 4, true},
                         {parents, (size_t)n * 4, false},
                         {children, (size_t)n * 4, false},
                         {lengths, (size_t)n * 4, false}};
    if ((st = check_ranges(what, all)) != FL_OK) return st;
    host::LaunchContext ctx;
    if ((st = host::launch_context(static_cast<cudaStream_t>(stream), &ctx)) != FL_OK) return st;
    PagesParams p = pages_params(cache, refs, lengths, workspace, ctx.range);
    p.parents = parents, p.children = children, p.n = n;
    if ((st = launch_pages<true>(what, p, ctx, static_cast<cudaStream_t>(stream))) != FL_OK) return st;
    CopyParams c = {};
    c.cache[0] = static_cast<uint8_t*>(cache->k_cache), c.cache[1] = static_cast<uint8_t*>(cache->v_cache);
    c.scale[0] = cache->k_scale, c.scale[1] = cache->v_scale;
    c.page_table = cache->page_table, c.refs = refs, c.lengths = lengths, c.parents = parents, c.children = children;
    c.table_stride = cache->table_stride, c.row_bytes = (long long)cache->heads * cache->head_dim;
    c.heads = cache->heads, c.n_seqs = cache->n_seqs, c.table_pages = cache->table_pages;
    c.n_pages = cache->n_pages, c.page_size = cache->page_size;
    return host::launched(host::launch(fl_kv_fork_copy_kernel, dim3((unsigned)n, kSlices), kCopyThreads, 0, ctx.pdl,
                                       static_cast<cudaStream_t>(stream), c),
                          what);
}

extern "C" fl_status fl_kv_compact(const fl_kv_pages* cache, const int* start, const int* accepted, int most, void* stream) {
    using namespace fl;
    const char* what = "fl_kv_compact";
    fl_status st;
    if ((st = check_table(what, cache)) != FL_OK) return st;
    if ((st = check_cache(what, cache)) != FL_OK) return st;
    if (most < 0) return fail(FL_ERR_INVALID_ARG, "%s: most must not be negative", what);
    if (most == 0) return host::ok();
    if ((st = check_ints(what, start)) != FL_OK) return st;
    if ((st = check_ints(what, accepted)) != FL_OK) return st;
    const size_t places = (size_t)cache->n_pages * cache->page_size * cache->heads;
    const Range all[] = {{cache->k_cache, places * cache->head_dim, true},
                         {cache->v_cache, places * cache->head_dim, true},
                         {cache->k_scale, places * 4, true},
                         {cache->v_scale, places * 4, true},
                         {cache->page_table, table_bytes(cache), false},
                         {start, (size_t)cache->n_seqs * 4, false},
                         {accepted, (size_t)cache->n_seqs * most * 4, false}};
    if ((st = check_ranges(what, all)) != FL_OK) return st;
    host::LaunchContext ctx;
    if ((st = host::launch_context(static_cast<cudaStream_t>(stream), &ctx)) != FL_OK) return st;
    CompactParams p = {};
    p.cache[0] = static_cast<uint8_t*>(cache->k_cache), p.cache[1] = static_cast<uint8_t*>(cache->v_cache);
    p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
    p.page_table = cache->page_table, p.start = start, p.accepted = accepted;
    p.table_stride = cache->table_stride, p.row_bytes = (long long)cache->heads * cache->head_dim;
    p.heads = cache->heads, p.most = most, p.table_pages = cache->table_pages;
    p.n_pages = cache->n_pages, p.page_size = cache->page_size, p.range = ctx.range;
    const bool wide = p.row_bytes % 16 == 0;
    const long long cols = 2 * p.row_bytes / (wide ? 16 : 8) + 2 * p.heads;
    if (cols > 65535ll * kMoveThreads) return fail(FL_ERR_UNSUPPORTED, "%s: too many heads", what);
    const dim3 grid((unsigned)cache->n_seqs, (unsigned)((cols + kMoveThreads - 1) / kMoveThreads));
    const cudaError_t e =
        wide ? host::launch(fl_kv_compact_kernel<uint4>, grid, kMoveThreads, 0, ctx.pdl, static_cast<cudaStream_t>(stream), p)
             : host::launch(fl_kv_compact_kernel<uint2>, grid, kMoveThreads, 0, ctx.pdl, static_cast<cudaStream_t>(stream), p);
    return host::launched(e, what);
}
