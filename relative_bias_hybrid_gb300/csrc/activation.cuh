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

// 2^x with results down to 2^-149.
__device__ __forceinline__ float wide_exp2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// kExact: for fp32 outputs, to a few units of the last place of the result, whatever its size; else for
// bf16 outputs, whose rounding is up to 2^-8 of the value: GELU within 1.5e-7 |v| / 2 (measured: within
// 0.36% of the value down to v = -6; values beyond, below 6e-9, keep fewer digits, and (1 + erf) / 2 in
// fp32 none), SILU within (4 + 1.2 |v|) 2^-23 of the value and 0 below 2^-126.
template <int kAct, bool kExact = false>
__device__ __forceinline__ float activate(float v) {
    if (kAct == INKATTN_ACT_RELU) return v <= 0.f ? 0.f : v;      // (a NaN stays one)
    if (kExact && kAct == INKATTN_ACT_GELU) {
        // v erfc(-v / sqrt 2) / 2 from h = erfc(|v| / sqrt 2) / 2 = 2^(-v^2 log2(e) / 2) t P(t) with t = 1 / (1 +
        // |v| / (2 sqrt 2)): P, of degree 8, is a fit of our own to exp(x^2) erfc(x) / (2 t), within 4.3e-8 of
        // the value for |v| up to 14 (and h is below 2^-141 beyond).  (erfcf in its place, whose two cases
        // diverge: 8192 x 512 x 4096 91 us where this takes 55 and the short form 45; 777 x 1000 x 1021 11.3,
        // 10.0 and 9.4.)
        const float t = reciprocal(fmaf(0.35355339f, fabsf(v), 1.f));
        float q = -0.0295190122f;
        q = fmaf(q, t, 0.14221178f);
        q = fmaf(q, t, -0.24344264f);
        q = fmaf(q, t, 0.138852909f);
        q = fmaf(q, t, -0.0131878322f);
        q = fmaf(q, t, 0.101290286f);
        q = fmaf(q, t, 0.121565387f);
        q = fmaf(q, t, 0.14118579f);
        q = fmaf(q, t, 0.14104332f);
        const float h = q * t * wide_exp2(v * v * -0.72134752f);
        return v > 0.f ? fmaf(-fminf(v, 15.f), h, v) : v * h;
    }
    if (kExact && kAct == INKATTN_ACT_SILU) {
        // (e is at most 1: nothing overflows.  8192 x 512 x 4096 44 us, the short form 38.)
        const float e = expf(-fabsf(v));
        return (v > 0.f ? v : v * e) * reciprocal(1.f + e);
    }
    if (kAct == INKATTN_ACT_GELU) {
        // v (1 + erf(x)) / 2 at x = v / sqrt 2, from erfc(|x|) by Abramowitz and Stegun, formula
        // 7.1.26: within 1.5e-7, without a branch (erff diverges within a warp, and its 32
        // copies in the epilogue spilled: 12.5 us for 777 x 1000 x 1021 where this took 9.6).
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
