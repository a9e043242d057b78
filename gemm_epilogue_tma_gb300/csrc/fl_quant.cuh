// Shared by the quantising kernels: the largest magnitude of 16-bit vectors
// (a NaN or an infinity shows in it) and the conversion of one 16-bit value.
#pragma once

#include "fl_common.cuh"

namespace fl {

// Bit patterns of the dtype.
template <int DT>
struct Bits16 {
    static constexpr uint32_t kInf = DT == DT_F16 ? 0x7c00u : 0x7f80u;
};

// Largest of the packed pairs' magnitudes, NaN if one is a NaN.
template <int DT>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == DT_F16)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    return r;
}

// Largest magnitude of 8 values, in both halves of the result.
template <int DT>
__device__ __forceinline__ uint32_t absmax8(const uint4& v) {
    const uint32_t m = absmax2<DT>(absmax2<DT>(v.x, v.y), absmax2<DT>(v.z, v.w));
    return absmax2<DT>(m, __funnelshift_l(m, m, 16));
}

}  // namespace fl
