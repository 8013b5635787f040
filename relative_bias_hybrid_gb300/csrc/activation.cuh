// activation.cuh -- the activations of the linear layers and the experts' products.
#pragma once

#include "common.cuh"

namespace inkattn {

// The unit's own 1 / x, within one unit of the last place; results below 2^-126 are 0.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int kAct>
__device__ __forceinline__ float activate(float v) {
    if (kAct == INKATTN_ACT_RELU) return v <= 0.f ? 0.f : v;      // (a NaN stays one)
    if (kAct == INKATTN_ACT_GELU) {
        // v (1 + erf(x)) / 2 at x = v / sqrt 2, from erfc(|x|) by Abramowitz and Stegun, formula
        // 7.1.26: within 1.5e-7, without a branch (erff diverges within a warp, and its 32
        // copies in the epilogue spilled: 12.5 us for 777 x 1000 x 1021 where this takes 9.6).
        // The formula's exp(-x^2) is 2^(-v^2 log2(e) / 2).
        const float t = reciprocal(fmaf(0.3275911f * 0.70710678f, fabsf(v), 1.f));
        const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f), 0.5f * 1.421413741f),
                                         0.5f * -0.284496736f), 0.5f * 0.254829592f);
        const float half_erfc = p * fast_exp2(v * v * -0.72134752f);
        // (half_erfc is 0 from v = 15 on; the bound keeps infinity from being multiplied by it)
        return v > 0.f ? fmaf(-fminf(v, 15.f), half_erfc, v) : v * half_erfc;
    }
    if (kAct == INKATTN_ACT_SILU) return v * reciprocal(1.f + fast_exp2(v * -1.44269504f));
    return v;
}

}  // namespace inkattn
