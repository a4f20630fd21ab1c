// The activations of the gated feed-forward block, for the kernels that form act(gate) * up.
#pragma once

#include "vae_types.cuh"

namespace vae {

// 1 / (1 + e^-z) in two approximate instructions (2^-22 relative beside the rounding of z log2 e; under e^-87 it is 0).
__device__ __forceinline__ float logistic(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// act(g), and its derivative.
template <int kAct>
__device__ __forceinline__ float act_value(float g) {
    if constexpr (kAct == VAE_ACT_GELU) return 0.5f * g * (1.f + erff(g * 0.70710678118654752440f));
    const float z = kAct == VAE_ACT_SILU ? g : 1.59576912160573071176f * (g + 0.044715f * g * g * g);
    return g * logistic(z);  // (1 + tanh(z / 2)) / 2
}
template <int kAct>
__device__ __forceinline__ float2 act_both(float g) {
    if constexpr (kAct == VAE_ACT_GELU) {
        const float cdf = 0.5f * (1.f + erff(g * 0.70710678118654752440f));
        return make_float2(g * cdf, cdf + g * 0.39894228040143267794f * __expf(-0.5f * g * g));
    }
    if constexpr (kAct == VAE_ACT_SILU) {
        const float s = logistic(g);
        return make_float2(g * s, s * (1.f + g * (1.f - s)));
    }
    // the slope's g z' (1 - s) at |g| <= 16: beyond, s is exactly 0 or 1 and so is the slope, but g z' grows as g^3 and would
    // meet 1 - s = 0, or s = 0, as an infinity
    const float z = 1.59576912160573071176f * (g + 0.044715f * g * g * g), s = logistic(z);
    const float h = fminf(fmaxf(g, -16.f), 16.f), dz = 1.59576912160573071176f * (1.f + 0.134145f * h * h);
    return make_float2(g * s, s * (1.f + h * dz * (1.f - s)));
}

}  // namespace vae
