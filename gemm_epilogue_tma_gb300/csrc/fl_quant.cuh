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

// Larger of the packed pairs' magnitudes, NaN if one is a NaN. (The sign of the
// result means nothing: mask it when done.)
template <int DT>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == DT_F16)
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int DT>
__device__ __forceinline__ uint32_t absmax8(const uint4& v) {
    return absmax2<DT>(absmax2<DT>(v.x, v.y), absmax2<DT>(v.z, v.w));
}

// Magnitude of the larger half, as 16 bits.
template <int DT>
__device__ __forceinline__ uint32_t absmax_halves(uint32_t m) {
    return absmax2<DT>(m, __funnelshift_l(m, m, 16)) & 0x7fffu;
}

// 1 / x within one unit in the last place; infinite for the smallest subnormals.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace fl
