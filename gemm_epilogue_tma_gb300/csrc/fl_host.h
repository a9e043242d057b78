// Host services of fl_host.cu for the entry points that live in other
// translation units: errors, the current device, argument checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/fusedlin.h"

namespace fl {
namespace host {

constexpr int kMaxDevices = 64;  // (allow_smem keeps one bit for each)

// Records the message for fl_last_error() and returns the status.
fl_status fail(fl_status s, const char* fmt, ...);
fl_status ok();

// What a launch on `stream` needs of the current device: its SM count, the
// stream's status word (bounded waits) and range word (indexes a kernel found
// outside their tables), and the launch options.
struct LaunchContext {
    int device;
    int sms;
    int* status;
    int* range;
    int pdl;
    unsigned long long timeout_ns;
};
fl_status launch_context(cudaStream_t stream, LaunchContext* ctx);

// Counts a launch and turns the launch call's result into a status.
fl_status launched(cudaError_t e, const char* what);

// Null and 16-byte alignment check of one pointer.
fl_status check_ptr(const char* name, const void* p, bool required);
bool overlap(const void* a, size_t na, const void* b, size_t nb);
// Whether two strided matrices of `elem`-byte elements whose spans overlap share
// no element because their rows interleave: the same row stride, and b's
// columns beside a's within it.
inline bool apart(const void* a, long long a_row, long long a_width, const void* b, long long b_row, long long b_width,
                  int elem) {
    if (a_row != b_row || a_row <= 0 || a_width > a_row || b_width > b_row) return false;
    const long long bytes = (long long)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a));
    if (bytes % elem != 0) return false;
    const long long d = ((bytes / elem) % a_row + a_row) % a_row;
    return d >= a_width && a_row - d >= b_width;
}
inline bool valid_dtype(int dt) { return dt == FL_F16 || dt == FL_BF16; }

// Strides (elements) of a [rows, heads, head_dim] tensor of 16-bit elements that is
// read or written in 16-byte vectors: multiples of 8, not negative, and for an
// output no two elements at one place (a row's heads lie inside its stride, or the
// rows inside a head's).
fl_status check_heads(const char* what, const char* name, int rows, int heads, int head_dim, long long row, long long head,
                      bool output);
// Its extent in bytes.
inline size_t span_heads(int rows, int heads, int head_dim, long long row, long long head) {
    return ((size_t)(rows - 1) * (size_t)row + (size_t)(heads - 1) * (size_t)head + (size_t)head_dim) * 2;
}

// Tensor map of a row-major [outer, inner] matrix of 16-bit elements (fp16 or
// bf16 by dt) or of bytes, box {box_inner, box_outer}, 128-byte swizzle, zero
// fill out of range.
fl_status encode_matrix(CUtensorMap* m, int dt, int elem_bytes, const void* ptr, uint64_t inner, uint64_t outer,
                        uint32_t box_inner, uint32_t box_outer);

// Tensor map of a [rows, heads, dim] tensor of 16-bit elements with contiguous
// channels: coordinates (channel, head, row), boxes of 64 channels of box_rows rows
// of one head, 128-byte swizzle, zero fill out of range.
fl_status encode_heads(CUtensorMap* m, int dt, const void* ptr, uint64_t dim, uint64_t heads, uint64_t rows,
                       uint64_t head_stride, uint64_t row_stride, uint32_t box_rows);

// Tensor map of the codes of a paged cache [pages, page_size, heads, dim] bytes, dim a
// multiple of 16: coordinates (channel, head, row in the page, page), boxes of
// `box_channels` (64 or 128) channels of box_rows rows of one head, as they are or with the
// swizzle of that width, zero fill out of range.
fl_status encode_pages(CUtensorMap* m, const void* ptr, uint64_t dim, uint64_t heads, uint64_t page_size, uint64_t pages,
                       uint32_t box_channels, uint32_t box_rows, bool swizzle);

// Lets `kern` use `bytes` of dynamic shared memory on `device`; asked of the
// runtime once per device (`done`: its bit is set).
template <typename Kern>
cudaError_t allow_smem(Kern kern, int bytes, int device, std::atomic<unsigned long long>& done) {
    if (done.load(std::memory_order_relaxed) >> device & 1) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(1ull << device, std::memory_order_relaxed);
    return e;
}

// cudaLaunchKernelEx with the programmatic-dependency attribute of the library's launches.
template <typename Kern, typename... Args>
cudaError_t launch(Kern kern, dim3 grid, int threads, size_t smem, int pdl, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = pdl;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The same in clusters of `cluster` CTAs along x.
template <typename Kern, typename... Args>
cudaError_t launch_cluster(Kern kern, dim3 grid, int threads, size_t smem, int pdl, int cluster, cudaStream_t stream,
                           const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute a[2];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = pdl;
    a[1].id = cudaLaunchAttributeClusterDimension;
    a[1].val.clusterDim.x = (unsigned)cluster, a[1].val.clusterDim.y = 1, a[1].val.clusterDim.z = 1;
    cfg.attrs = a;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace host

// The argument checks of fl_rope and fl_kv_write alone (fl_layer_attach_cache).
fl_status check_rope(const fl_rope_desc* desc);
fl_status check_kv_write(const fl_kv_desc* desc);

}  // namespace fl
