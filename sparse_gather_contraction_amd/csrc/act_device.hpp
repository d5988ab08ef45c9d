// act_device.hpp — the activation functions of the channel products and their slopes.
#pragma once

#include "common.hpp"
#include "disco.h"

namespace disco {

// 1/2 + an odd function h of v, as v times a polynomial in v^2 on [-L, L], 1/2 + h(L) = 1 beyond.  The coefficients are a
// least-maximum fit of h(v) / v over t = 2 v^2 / L^2 - 1 in fp64, subject to the value at L; a NaN stays one.  With the last
// product rounded before the sum (no fma) the ends are 0 and 1 exactly.  In fp32 arithmetic off by 2.4e-7 (the normal
// distribution function) and 5.1e-7 (the slope of gelu) at most, anywhere, in two thirds of the time that an exponential and a
// reciprocal take (the 8-bit form steps by 1/127, fp16 by 5e-4 of 1).
template <int N>
__device__ __forceinline__ float half_and_odd(float v, float L, float scale, const float (&c)[N])
{
#pragma clang fp contract(off)
    const float x = __builtin_elementwise_maximum(__builtin_elementwise_minimum(v, L), -L);
    const float t = __builtin_fmaf(x * x, scale, -1.0f);
    float p = c[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) {
        float k = c[i];
        asm("" : "+s"(k));   // in a scalar register: as a literal, a quarter of the sums would take a move of their own
        p = __builtin_fmaf(p, t, k);
    }
    const float h = p * x;
    return h + 0.5f;
}

__device__ __forceinline__ float normal_cdf(float v)
{
    constexpr float c[14] = {0.137932017f, -0.0686848387f, 0.0505928136f, -0.0401603915f, 0.0318186842f, -0.0241475701f, 0.0174531564f,
                             -0.0122796884f, 0.00762281241f, -0.00349970278f, 0.00188006158f, -0.00176295277f, 0.000951673777f,
                             -0.000155099362f};
    return half_and_odd(v, 5.125f, 0.07614515f, c);
}

__device__ __forceinline__ float gelu_slope(float v)
{
    constexpr float c[16] = {0.125845447f, -0.0639348626f, 0.0513828993f, -0.0502946228f, 0.0556100719f, -0.0642657354f, 0.0726433396f,
                             -0.0718892291f, 0.0596861281f, -0.0565041192f, 0.0597264618f, -0.03331545f, 0.00105434807f,
                             -0.00697237113f, 0.0174371265f, -0.00732053956f};
    return half_and_odd(v, 5.625f, 0.06320988f, c);
}

__device__ __forceinline__ float logistic(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

template <int ACT>
__device__ __forceinline__ float act_value(float v)
{
    if constexpr (ACT == DISCO_ACT_GELU) {
        return v * normal_cdf(v);
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
        return gelu_slope(v);
    } else if constexpr (ACT == DISCO_ACT_SILU) {
        const float s = logistic(v);
        return s * __builtin_fmaf(v, 1.0f - s, 1.0f);
    } else {
        return 1.0f;
    }
}

}  // namespace disco
