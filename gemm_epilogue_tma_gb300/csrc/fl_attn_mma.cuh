// What the attention kernels on the tensor cores share: waits without a call, groups of
// MMAs issued by an elected lane, the descriptor of an operand whose rows are k.
#pragma once

#include "fl_common.cuh"

namespace fl {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The bounded waits of fl_common.cuh without a call: a function call in a kernel
// that moves registers between its warps (setmaxnreg) cannot be compiled.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, int* status, unsigned long long timeout_ns, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 0) {
            if (*reinterpret_cast<volatile int*>(status) != 0) return false;
            if (globaltimer_ns() - t0 > timeout_ns) {
                atomicCAS(status, 0, kStatusTimeout | (where << 8));
                return false;
            }
        }
    }
}
__device__ __forceinline__ void drain_here(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 20000000ull) {}
}

// Four MMAs of 16 k each by an elected lane of a converged warp, A and B 32 bytes
// further along their swizzled rows from one to the next.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r, x1, x2, x3, l1, l2, l3;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
        "elect.sync r|p, 0xffffffff;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "add.u32 x1, %1, 2;\n\tadd.u32 x2, %1, 4;\n\tadd.u32 x3, %1, 6;\n\t"
        "add.u32 l1, %2, 2;\n\tadd.u32 l2, %2, 4;\n\tadd.u32 l3, %2, 6;\n\t"
        "mov.b64 a0, {%1, %3};\n\tmov.b64 a1, {x1, %3};\n\tmov.b64 a2, {x2, %3};\n\tmov.b64 a3, {x3, %3};\n\t"
        "mov.b64 b0, {%2, %3};\n\tmov.b64 b1, {l1, %3};\n\tmov.b64 b2, {l2, %3};\n\tmov.b64 b3, {l3, %3};\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %4, q;\n\t"
        "setp.eq.u32 q, 0, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %4, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %4, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %4, q;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
        : "memory");
}
// The same with A in tensor memory (8 columns of 16 k) and B of 16 keys, 2048 bytes, from one to the next.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r, x1, x2, x3, l1, l2, l3;\n\t.reg .b64 b0, b1, b2, b3;\n\t"
        "elect.sync r|p, 0xffffffff;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "add.u32 x1, %1, 8;\n\tadd.u32 x2, %1, 16;\n\tadd.u32 x3, %1, 24;\n\t"
        "add.u32 l1, %2, 128;\n\tadd.u32 l2, %2, 256;\n\tadd.u32 l3, %2, 384;\n\t"
        "mov.b64 b0, {%2, %3};\n\tmov.b64 b1, {l1, %3};\n\tmov.b64 b2, {l2, %3};\n\tmov.b64 b3, {l3, %3};\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, q;\n\t"
        "setp.eq.u32 q, 0, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x1], b1, %4, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x2], b2, %4, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x3], b3, %4, q;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 r;\n\telect.sync r|p, 0xffffffff;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Descriptor of an MN-major operand with the 128-byte swizzle:
// rows of 64 elements (128 bytes) along N, one per k; 1024 bytes from eight
// k to the next, `chunk` bytes from 64 elements of N to the next.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t chunk) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(chunk >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
constexpr uint32_t kBMajorN = 1u << 16;  // instruction descriptor: B is MN-major

}  // namespace fl
