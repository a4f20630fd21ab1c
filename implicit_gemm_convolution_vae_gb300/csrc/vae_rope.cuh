// The angles of rotary positions, for the kernels that turn pairs by them.
//
// The angle of pair p at position t is 2 pi t f_p with f_p turns per position.
// f_p comes from the host in two floats (hi + lo, 48 bits), so t f_hi is split
// exactly by one fma into whole turns and a fraction, t f_lo is added to the
// fraction, and sincospi of twice the fraction follows: far positions lose no
// digits and no 64-bit arithmetic runs on the device.
#pragma once

#include "vae_common.cuh"

namespace vae {

// Turns (a, b) by (cos, sin).
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
    const float x = a * cs.x - b * cs.y;
    b = a * cs.y + b * cs.x;
    a = x;
}

// (cos, sin) of pair `pr` at a position.
__device__ __forceinline__ float2 rope_cos_sin(const vae_rope_plan& plan, int pr, float pos) {
    // whole turns + fraction of pos * hi (the fma's product is exact), then the rest
    const float hi = plan.turns_hi[pr];
    const float whole = rintf(pos * hi);
    const float frac = fmaf(pos, hi, -whole) + pos * plan.turns_lo[pr];
    float sn, c;
    sincospif(2.f * frac, &sn, &c);
    return make_float2(c, sn);
}

}  // namespace vae
