// linear.hpp — launch descriptors of the 8-bit form and the channel products (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "linear_plan.hpp"

namespace disco {

// element types: 0 = fp32, 1 = bf16, 2 = fp16
struct FormLaunch {
    const void *x = nullptr;       // writer: input; reader: null
    void *out = nullptr;           // reader: output
    int8_t *q = nullptr;           // the form
    float *scale = nullptr;
    int8_t *kq = nullptr;          // writer: the checkpoint, or null
    float *kscale = nullptr;
    int32_t dtype = 0, act = 0;
    int64_t N = 0, D = 0, M = 0;
};

hipError_t launch_quantize_i8(const FormLaunch &a, hipStream_t stream);
hipError_t launch_dequantize_i8(const FormLaunch &a, hipStream_t stream);

// y = q w^T with scales: P points in planes of M (M = 1: rows), C padded to Cp, Co outputs
struct LinearLaunch {
    const int8_t *q = nullptr;
    const float *scale = nullptr;
    const int8_t *w = nullptr;
    const float *wscale = nullptr;
    const void *bias = nullptr;    // fp32, or null
    void *y = nullptr;
    int32_t dtype = 0;
    int64_t P = 0, M = 1, Cp = 0, Co = 0;
};

hipError_t launch_linear_i8(const LinearLaunch &a, hipStream_t stream);

struct LinearBwdLaunch {
    const void *gy = nullptr;      // (N, Co, M), 16 bits
    const int8_t *q = nullptr;     // input: w (Co, Cp); weight: the form of x (P, Cp)
    const float *scale = nullptr;
    const int8_t *kept = nullptr;  // input: the activation function's checkpoint (P, Cp), or null
    const float *kept_scale = nullptr;
    void *out = nullptr;           // input: gx (N, C, M); weight: dw (Co, C)
    void *db = nullptr;            // weight: (Co), or null
    float *workspace = nullptr;    // weight, more than one split: [splits][Co][C], then [splits][Co]
    int32_t dtype = 0, act = 0, splits = 1;
    int64_t P = 0, M = 1, C = 0, Cp = 0, Co = 0;
};

// The input's gradient with the weights in registers: which calls, and the launch (nt: stores past the caches).
bool bwd_stays(const LinearBwdLaunch &a);
hipError_t launch_linear_bwd_stay(const LinearBwdLaunch &a, bool nt, hipStream_t stream);

hipError_t launch_linear_bwd_input(const LinearBwdLaunch &a, hipStream_t stream);
hipError_t launch_linear_bwd_weight(const LinearBwdLaunch &a, hipStream_t stream);

}  // namespace disco
