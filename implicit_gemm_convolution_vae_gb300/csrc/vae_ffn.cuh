// The activations of the gated feed-forward block, for the kernels that form act(gate) * up.
#pragma once

#include "vae_types.cuh"

namespace vae {

__device__ __forceinline__ float exp2_near(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float inverse_near(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-z) in two approximate instructions (2^-22 relative beside the rounding of z log2 e; under e^-87 it is 0).
__device__ __forceinline__ float logistic(float z) { return inverse_near(1.f + exp2_near(z * -1.4426950408889634f)); }

// Phi(g), the normal distribution function, and e^(-g^2/2). The tail beyond a = |g| is e^(-a^2/2) times a smooth function
// of it, here t P(t) with t = 1 / (1 + 0.3 a) and P of degree 7 fitted for the least relative error over 0 <= a <= 14.5
// (1.64e-7). In all 2^-20 and 2^-23 g^2 relative, where 0.5 (1 + erf) cancels for g < 0: a tenth of it lost at -5, all
// at -5.6. (erfcf instead: 16384 tokens of 1152 x 4608 386 us, the gradient 790, where erff took 351 and 728.)
__device__ __forceinline__ float2 normal(float g) {
    const float t = inverse_near(fmaf(0.3f, fabsf(g), 1.f)), e = exp2_near(g * g * -0.72134752044448170368f);
    float p = fmaf(0.03542390465736389f, t, -0.15615932643413544f);
    p = fmaf(p, t, 0.2045585662126541f);
    p = fmaf(p, t, -0.052035871893167496f);
    p = fmaf(p, t, 0.12769284844398499f);
    p = fmaf(p, t, 0.10017560422420502f);
    p = fmaf(p, t, 0.12071219086647034f);
    p = fmaf(p, t, 0.11963200569152832f);
    const float tail = p * t * e;
    return make_float2(g < 0.f ? tail : 1.f - tail, e);
}

// act(g), and its derivative.
template <int kAct>
__device__ __forceinline__ float act_value(float g) {
    if constexpr (kAct == VAE_ACT_GELU) return g * normal(g).x;
    const float z = kAct == VAE_ACT_SILU ? g : 1.59576912160573071176f * (g + 0.044715f * g * g * g);
    return g * logistic(z);  // (1 + tanh(z / 2)) / 2
}
template <int kAct>
__device__ __forceinline__ float2 act_both(float g) {
    if constexpr (kAct == VAE_ACT_GELU) {
        const float2 n = normal(g);
        return make_float2(g * n.x, fmaf(g * 0.39894228040143267794f, n.y, n.x));
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
