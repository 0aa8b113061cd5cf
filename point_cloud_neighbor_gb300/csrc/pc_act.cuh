// pc_act.cuh -- the activations of group norm and the gated projection, and
// their derivatives, in float32.
#pragma once

#include "pointcloud.h"

#include <cuda_runtime.h>

#include <type_traits>

namespace pcn {

__device__ __forceinline__ float approx_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float approx_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float LOG2_E = 1.4426950408889634f;

// s(z) = 1 / (1 + exp(-z)); the reciprocal of a number from 1 on, off by 2^-23.
// FAST, for results that are rounded to bfloat16: exp as a power of 2 whose exponent is
// rounded once: off by up to 2^-21 (|z| + 2) relative.
template <bool FAST>
__device__ __forceinline__ float logistic(float z) {
    return approx_rcp(1.0f + (FAST ? approx_ex2(-LOG2_E * z) : expf(-z)));
}

// The normal distribution's cumulative function and e = exp(-z^2 / 2), the far negative
// side with its relative accuracy.  Not FAST: by erfc.  FAST, for results that are rounded
// to bfloat16:
//   erfc(x) = (a1 t + ... + a7 t^7) exp(-x^2),  t = 1 / (1 + p x),  x = |z| / sqrt(2),
// the form of Hastings's approximations (formula 7.1.26 of Abramowitz and Stegun's Handbook
// of Mathematical Functions), with coefficients fitted here by linear programming so that
// the largest relative error over x <= 9.5 (beyond, e is below float32) is least: 5e-7,
// with the roundings (of the exponent, mostly) 2e-6 from z = -5 on and 8e-6 at the end.  The
// printed formula's is absolute (1.5e-7), which leaves 0.7% at z = -7.  (With a term less
// 3.7e-6, which float32 sums of the derivative over many points show.)  It takes half the
// instructions of erff and shares the exponential with the derivative.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    if (!FAST) {
        e = expf(-0.5f * z * z);
        return 0.5f * erfcf(-0.70710678118654752f * z);
    }
    const float t = approx_rcp(fmaf(fabsf(z), 0.37339323f * 0.70710678f, 1.0f));
    e = approx_ex2(-0.5f * LOG2_E * z * z);
    float p = fmaf(0.5f * -0.13863525f, t, 0.5f * 0.4069617f);
    p = fmaf(p, t, 0.5f * -0.15283303f);
    p = fmaf(p, t, 0.5f * 0.29764012f);
    p = fmaf(p, t, 0.5f * 0.16079962f);
    p = fmaf(p, t, 0.5f * 0.21569888f);
    p = fmaf(p, t, 0.5f * 0.21036738f);
    const float q = p * t * e;
    return z < 0.0f ? q : 1.0f - q;
}

// act(z).  The activation is a template parameter: a switch for every value keeps
// the values of a thread from being computed side by side (the gated projection of 16,384 x
// 384 x 1024 took 68 instead of 29 us).
template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == PC_ACT_SILU) return z * logistic<FAST>(z);
    if (ACT == PC_ACT_GELU) {
        float e;
        return z * normal_cdf<FAST>(z, e);
    }
    if (ACT == PC_ACT_RELU) return z > 0.0f || z != z ? z : 0.0f;  // (a NaN stays)
    if (ACT == PC_ACT_SIGMOID) return logistic<FAST>(z);
    return z;
}

// act(z) and act'(z)
template <int ACT, bool FAST>
__device__ __forceinline__ float act_both(float z, float &slope) {
    if (ACT == PC_ACT_SILU) {
        const float s = logistic<FAST>(z);
        slope = s * fmaf(z, 1.0f - s, 1.0f);
        return z * s;
    }
    if (ACT == PC_ACT_GELU) {
        constexpr float N = 0.39894228040143268f;  // 1 / sqrt(2 pi)
        float e;
        const float c = normal_cdf<FAST>(z, e);
        slope = fmaf(z * N, e, c);
        return z * c;
    }
    if (ACT == PC_ACT_RELU) {
        slope = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
        return z > 0.0f || z != z ? z : 0.0f;
    }
    if (ACT == PC_ACT_SIGMOID) {
        const float s = logistic<FAST>(z);
        slope = s * (1.0f - s);
        return s;
    }
    slope = 1.0f;
    return z;
}

// f(activation as a compile-time constant)
template <class F>
__device__ __forceinline__ void act_switch(int act, F f) {
    switch (act) {
        case PC_ACT_SILU: f(std::integral_constant<int, PC_ACT_SILU>{}); break;
        case PC_ACT_GELU: f(std::integral_constant<int, PC_ACT_GELU>{}); break;
        case PC_ACT_RELU: f(std::integral_constant<int, PC_ACT_RELU>{}); break;
        case PC_ACT_SIGMOID: f(std::integral_constant<int, PC_ACT_SIGMOID>{}); break;
        default: f(std::integral_constant<int, PC_ACT_NONE>{}); break;
    }
}

}  // namespace pcn
