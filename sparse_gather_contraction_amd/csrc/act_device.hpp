// act_device.hpp — the activation functions of the channel products and their slopes.
#pragma once

#include "common.hpp"
#include "disco.h"

namespace disco {

// The normal distribution's lower tail, Phi(-t) = e^(-t^2/2) R(t): e and the polynomial p = R(t) in w = 1 / (1 + 0.34 t) at
// t = |v|, up to 14.5 where e is 0 in fp32.  The coefficients are a least-maximum fit on [0, 13.2] in fp64 of the error relative
// to R, weighted by 1 / (1 + t^2 / 8): off by 9.1e-8 (1 + t^2 / 8) of R.  With e's argument rounded (three roundings of
// t^2 / 2) the tail is off by a part in 2.4e6 near 0, 6e5 at 4 and 1e5 at 12: a point whose values all lie in it has a scale and codes
// as good as any other's.  A NaN stays one.  (1/2 plus an odd polynomial, off by 2.4e-7 of 1 anywhere, has no such tail and is
// hardly faster: the 8-bit form of 259200x2048 bf16 with gelu and a checkpoint, and two readers, 904 us against 921; input's
// gradients through its slope, off by 5.1e-7, 941 us against 934 at 2048 from 512.)
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

// Phi(v) + v phi(v): at -t e^(-t^2/2) (R(t) - t / sqrt(2 pi)), at t one less that.  The difference is R's error away from 0 at its
// one zero (t = 0.752), and as good as R where the tail is small.
__device__ __forceinline__ float gelu_slope(float v)
{
    const NormalTail n = normal_tail(v);
    const float z = n.e * __builtin_fmaf(n.t, -0.3989422804014327f, n.p);
    return v < 0.0f ? z : 1.0f - z;
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
