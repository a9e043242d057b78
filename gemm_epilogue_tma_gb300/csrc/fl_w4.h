// Declarations shared by the 4-bit product kernels.
#pragma once

#include <cstdint>

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
    float eps;
};

}  // namespace fl
