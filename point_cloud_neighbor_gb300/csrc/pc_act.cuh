// pc_act.cuh -- the activations of group norm and the gated projection, and
// their derivatives, in float32.
#pragma once

#include "pointcloud.h"

#include <cuda_runtime.h>

#include <type_traits>

namespace pcn {

// s(z) = 1 / (1 + exp(-z)).  FAST, for results that are rounded to bfloat16:
// the approximate exponential and quotient, off by up to 2^-21 (|z| + 2) relative.
template <bool FAST>
__device__ __forceinline__ float logistic(float z) {
    if (FAST) return __fdividef(1.0f, 1.0f + __expf(-z));
    return 1.0f / (1.0f + expf(-z));
}

// The normal distribution's cumulative function.  Not FAST: by erfc, so that
// the far negative side keeps its relative accuracy; FAST off by 2^-24 absolute.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z) {
    constexpr float R = 0.70710678118654752f;
    if (FAST) return fmaf(0.5f, erff(R * z), 0.5f);
    return 0.5f * erfcf(-R * z);
}

// act(z).  The activation is a template parameter: a switch for every value keeps
// the values of a thread from being computed side by side (a tile's epilogue took
// ten times as long).
template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == PC_ACT_SILU) return z * logistic<FAST>(z);
    if (ACT == PC_ACT_GELU) return z * normal_cdf<FAST>(z);
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
        const float c = normal_cdf<FAST>(z);
        const float e = FAST ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
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
