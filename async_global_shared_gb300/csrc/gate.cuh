// The activation of a gated block, its slope, and their constants.
//
// Both activations are act(g) = g s(w(g)) with the logistic function
// s(w) = 1 / (1 + exp(-w)) of a polynomial w(g) = g (c1 + c3 g^2):
//     silu  w = g;
//     gelu  w = 2 sqrt(2 / pi) (g + 0.044715 g^3), since (1 + tanh z) / 2 = s(2 z);
// so one instruction stream serves both, and
//     act'(g) = s + g s (1 - s) w'(g) = s (1 + g (1 - s) w'(g)),  w'(g) = c1 + 3 c3 g^2.
#pragma once

#include <cstdint>

#include "asyncpipe_gated.h"
#include "fp8_common.cuh"

namespace ap {

struct Gate {
    float e1, e3;  // c1 and c3 times log2(e): exp(-w) = 2^(-near (e1 + e3 near^2))
    float c1, c9;  // c1 and 3 c3, of w'
};

inline Gate gate_of(ap_activation act) {
    constexpr double kRoot = 0.79788456080286535588, kLog2e = 1.44269504088896340736;  // sqrt(2 / pi), log2(e)
    const double c1 = act == AP_ACT_GELU ? 2 * kRoot : 1, c3 = act == AP_ACT_GELU ? 2 * kRoot * 0.044715 : 0;
    return Gate{static_cast<float>(c1 * kLog2e), static_cast<float>(c3 * kLog2e), static_cast<float>(c1), static_cast<float>(3 * c3)};
}

// s(w(g)), by the hardware's approximations of 2^x and 1 / x (each within two
// units in the last place). Past +-128 both activations have s = 0 or 1 in 32 bits,
// so g enters no further: `low` is g down to -128 and what act multiplies with s (0
// there, at -infinity too), and the polynomial takes it up to 128, which keeps
// infinities out of it; NaN stays NaN. The exponential takes the roundings of its
// argument, at most three halves of a unit of w, so s is off by at most
// (8 + 3 |w|) 2^-24 of itself while it is a normal number, w above about -87.3. An s
// below 2^-126 comes out of the reciprocal as 0: act(g) is then 0, off by less than
// |g| 2^-126 (silu(-88) is -5.3e-37), and its slope 0, off by less than
// (1 + |g| w'(g)) 2^-126. (gated_grad.cu has the same for two values.)
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// act(g).
__device__ __forceinline__ float gate_value(const Gate& p, float g) {
    const float low = max_nan(g, -128.0f), near = min_nan(low, 128.0f);
    return low * rcp_approx(1.0f + exp2_approx(-near * fmaf(p.e3, near * near, p.e1)));
}

}  // namespace ap
