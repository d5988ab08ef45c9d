// act_device.hpp — the activation functions of the channel products and their slopes.
#pragma once

#include "common.hpp"
#include "disco.h"

namespace disco {

// Phi(-|v|), the normal distribution's tail, and e^(-v^2/2): erfc(z) = t (a1 + t (a2 + ...)) e^(-z^2) with
// t = 1 / (1 + p z) and z = |v| / sqrt 2, the five-term rational form of Hastings (Abramowitz and Stegun 7.1.26), off by
// 1.5e-7 at most.  That is 1/50000 of a step of the 8-bit form, and below the last place of a slope in fp16.
__device__ __forceinline__ float normal_tail(float v, float &e)
{
    const float z = __builtin_fabsf(v) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(z, 0.3275911f, 1.0f));
    e = __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);  // log2(e) / 2
    float p = __builtin_fmaf(t, 1.061405429f, -1.453152027f);
    p = __builtin_fmaf(t, p, 1.421413741f);
    p = __builtin_fmaf(t, p, -0.284496736f);
    p = __builtin_fmaf(t, p, 0.254829592f);
    return 0.5f * p * t * e;
}

__device__ __forceinline__ float logistic(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

template <int ACT>
__device__ __forceinline__ float act_value(float v)
{
    if constexpr (ACT == DISCO_ACT_GELU) {
        float e;
        const float tail = normal_tail(v, e);
        return v * (v >= 0.0f ? 1.0f - tail : tail);
    } else if constexpr (ACT == DISCO_ACT_SILU) {
        return v * logistic(v);
    } else {
        return v;
    }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float v)
{
    if constexpr (ACT == DISCO_ACT_GELU) {
        float e;
        const float tail = normal_tail(v, e), phi = v >= 0.0f ? 1.0f - tail : tail;
        return __builtin_fmaf(v * 0.39894228040143268f, e, phi);
    } else if constexpr (ACT == DISCO_ACT_SILU) {
        const float s = logistic(v);
        return s * __builtin_fmaf(v, 1.0f - s, 1.0f);
    } else {
        return 1.0f;
    }
}

}  // namespace disco
