// Declarations shared by the 4-bit product kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fl_host.h"
#ifdef __CUDACC__
#include "fl_common.cuh"
#endif

namespace fl {

// One product on a 4-bit weight, or (two weights) the SwiGLU gate/up pair.
struct W4Params {
    const uint16_t* x;         // [M, K]
    const uint16_t* gamma;     // [K] or null
    const uint8_t* q[2];       // [N, K / 2]
    const uint16_t* scales[2]; // [N, K / group]
    const uint8_t* zeros[2];   // [N, K / group] or null
    const uint16_t* bias;      // [N] or null
    const uint16_t* residual;  // [M, N] or null
    uint16_t* out;             // [M, N]
    int M, N, K, group, act;
    int slab;                  // decode kernel: rows of one slab of the grid, and whether
    bool halves;               // x * gamma is carried as two 16-bit numbers
    float eps;
};

// Decode kernel (fl_w4_rows.cu): few rows that fit in shared memory, with the RMSNorm prologue.
bool w4_few_rows(int M, int N, int K, bool dual);
bool w4_always_few(int M, int K);  // whatever N is
fl_status w4_rows(int dt, bool dual, const W4Params& p, const host::LaunchContext& ctx, cudaStream_t stream);

// Tile kernel (fl_w4_tile.cu): any number of rows; the RMSNorm prologue keeps the rows' scales in the workspace.
size_t w4_tile_workspace(int M, bool norm);
fl_status w4_tile(int dt, bool dual, const W4Params& p, void* workspace, const host::LaunchContext& ctx, cudaStream_t stream);

#ifdef __CUDACC__
// (a & mask) | bits as one instruction (the compiler makes two of it when both are immediates)
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

// The activations of the 4-bit products: GeLU (tanh form) and SiLU as
// v sigmoid(z) = v / (1 + 2^t), t = -z log2(e), z = 2 sqrt(2/pi) (v + 0.044715 v^3) or v,
// within 2^-18 of the value (the power of two's error grows with t: some
// 2^-20 at 24), and 0 where 2^t passes 2^126. The hardware tanh that act_apply takes is
// off by 2^-11 of the tanh, which is |v| 2^-12 of the product whatever is left
// of it: silu(-8) = -0.0027 could be off by 0.002. One special-function operation
// more a value: 2048 x 4096 x 4096 with SiLU 64.0 -> 65.4 us, FFN of 64 and 2048 rows equal.
__device__ __forceinline__ float w4_act(int act, float v) {
    if (act == ACT_RELU) return fmaxf(v, 0.0f);
    if (act == ACT_NONE) return v;
    const float a = -1.4426950408889634f, b = -2.302208198f;  // -log2(e), -2 sqrt(2 / pi) log2(e)
    const float t = act == ACT_GELU ? v * fmaf(0.044715f * b, v * v, b) : v * a;
    float p, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + p));
    return v * q;
}
#endif

}  // namespace fl
