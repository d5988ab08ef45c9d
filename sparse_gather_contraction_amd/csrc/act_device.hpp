// act_device.hpp — the activation functions of the channel products and their slopes.
#pragma once

#include "common.hpp"
#include "disco.h"

namespace disco {

// The normal distribution's lower tail, Phi(-t) = e^(-t^2/2) R(t): e and the polynomial p = R(t) in w = 1 / (1 + 0.34 t) at
// t = |v|, up to 14.5 where e is 0 in fp32.  The coefficients are a least-maximum fit on [0, 13.2] in fp64 of the error relative
// to R, weighted by 1 / (1 + t^2 / 8): off by 9.1e-8 (1 + t^2 / 8) of R.  With e's argument rounded (three roundings of
// t^2 / 2) the tail is off by a part in 2.4e6 near 0, 6e5 at 4 and 1e5 at 12: a point whose values all lie in it has a scale and codes
// as good as any other's.  A NaN stays one.
struct NormalTail {
    float t, e, p;
};

__device__ __forceinline__ NormalTail normal_tail(float v)
{
    constexpr float c[8] = {-6.47412016e-05f, 0.136969f, 0.124231048f, 0.173438743f, -0.0601831488f, 0.293716341f, -0.216521159f, 0.0484139621f};
    NormalTail r;
    r.t = __builtin_elementwise_minimum(__builtin_fabsf(v), 14.5f);
    const float w = __builtin_amdgcn_rcpf(__builtin_fmaf(r.t, 0.34f, 1.0f));
    r.p = c[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) {
        float k = c[i];
        asm("" : "+s"(k));   // in a scalar register: as a literal, some of the sums would take a move of their own
        r.p = __builtin_fmaf(r.p, w, k);
    }
    r.e = __builtin_amdgcn_exp2f(r.t * r.t * -0.7213475204444817f);
    return r;
}

// v Phi(v) = max(v, 0) - |v| Phi(-|v|).
__device__ __forceinline__ float gelu(float v)
{
    const NormalTail n = normal_tail(v);
    return __builtin_fmaf(-__builtin_fabsf(v), n.e * n.p, __builtin_elementwise_maximum(v, 0.0f));
}

// 1/2 + an odd function h of v, as v times a polynomial in v^2 on [-L, L], 1/2 + h(L) = 1 beyond.  The coefficients are a
// least-maximum fit of h(v) / v over t = 2 v^2 / L^2 - 1 in fp64, subject to the value at L; a NaN stays one.  With the last
// product rounded before the sum (no fma) the ends are 0 and 1 exactly.  In fp32 arithmetic off by 5.1e-7 at most, anywhere.
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
        return gelu(v);
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
