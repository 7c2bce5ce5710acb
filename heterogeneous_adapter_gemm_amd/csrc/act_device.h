// The gate's activations on the device, in fp32.
#pragma once

#include "common.h"
#include "rows.h"

namespace hagemm {

// e^v for the gates: the hardware's 2^x of v log2(e), the product's rounding error given back, so that a
// large v loses no more than a small one
__device__ __forceinline__ float exp_gate(float v) {
    constexpr float kLog2e = 1.44269504088896340736f, kLog2eRest = 1.92596299112661746887e-8f;
    const float t = v * kLog2e;
    const float rest = fmaf(v, kLog2eRest, fmaf(v, kLog2e, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    return fabsf(t) < 126.f ? fmaf(p, rest * 0.69314718055994530942f, p) : p;   // (beyond: 0, infinity, or next to them)
}

// silu(v) = v / (1 + e^-v); gelu(v) = v P(N(0, 1) <= v) = v erfc(-v / sqrt 2) / 2; gelu_tanh(v) = v / (1 + e^-2u),
// u = sqrt(2 / pi) (v + 0.044715 v^3), which is v (1 + tanh u) / 2 without its cancellation at negative v
template <int ACT>
__device__ __forceinline__ float activate(float v) {
    if constexpr (ACT == kActSilu) {
        return v / (1.f + exp_gate(-v));
    } else if constexpr (ACT == kActGelu) {
        return 0.5f * v * erfcf(v * -0.70710678118654752440f);
    } else if constexpr (ACT == kActGeluTanh) {
        const float u2 = -1.59576912160573071176f * fmaf(0.044715f * v * v, v, v);
        return v / (1.f + exp_gate(u2));
    } else {
        return v;
    }
}

}  // namespace hagemm
