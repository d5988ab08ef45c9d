// norm.hpp — launch descriptors of the norm, 8-bit and gradient kernels (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "norm_plan.hpp"

namespace disco {

typedef double part_t __attribute__((aligned(4)));   // a partial sum of dw: a workspace has fp32's alignment

// element types: 0 = fp32, 1 = bf16, 2 = fp16
struct NormLaunch {
    const void *x = nullptr;   // forward: x; backward: the stored sum h
    const void *r = nullptr;   // forward: residual or null; backward: gh or null
    const void *gy = nullptr;  // backward
    const void *w = nullptr;
    void *y = nullptr;         // forward: y or q; backward: gx
    void *h = nullptr;         // forward: the stored sum (with r)
    float *scale = nullptr;    // 8-bit output
    void *dw = nullptr;        // backward
    void *workspace = nullptr; // backward: as BwdPlan::bytes says
    int32_t dtype = 0;
    int32_t wf32 = 1;          // the weight (and dw) is fp32, else of the data type
    int64_t N = 0, D = 0, M = 0;
    float eps = 0;
    int32_t f8 = -1;           // -1: no 8-bit output, 0: e4m3, 1: e5m2
    int32_t group = 0;         // channels of one scale (8-bit output)
    int32_t ngroups = 1;
};

hipError_t launch_norm(const NormLaunch &a, hipStream_t stream);
hipError_t launch_norm_bwd(const NormLaunch &a, hipStream_t stream);

struct DequantLaunch {
    const uint8_t *q;
    const float *scale;
    void *out;
    int32_t dtype, f8;
    int64_t N, D, M;
    int32_t group, ngroups;
};

hipError_t launch_dequant(const DequantLaunch &a, hipStream_t stream);

// One run of a launch over many: `n` elements at `p`, written to `o` by the scaling pass.
struct GradTensor {
    const void *p;
    void *o;
    int64_t n;
    int32_t first;   // its first chunk in the launch
    int32_t dtype;
};

constexpr int kGradBatch = 120;     // runs a launch takes in its arguments (32 bytes each, below 4 KiB; 128 at most)
constexpr int kGradBlocks = 2048;   // workgroups of one norm launch (all a GPU holds), so partial sums it leaves
constexpr int kGradDirect = 2048;   // up to so many partial sums, each scaling workgroup adds them itself

struct GradBatch {
    GradTensor t[kGradBatch];
    int32_t count;
    int32_t chunks;
    int32_t chunk;   // elements of a chunk
    int32_t stream;  // loads and stores that the caches drop first
};

// Few elements: their chunks, done by one workgroup in one launch (5 bf16 tensors of 905 elements in all 6.0 against 8.7 us).
constexpr int kSmallChunks = 8;
constexpr int64_t kSmallElements = 16384, kSmallChunk = 8192;

struct GradSmall {
    GradTensor t[kSmallChunks];
    int32_t count;
};

// The sum of `g`'s squares to partial[0], its root to `norm`, and `out` (none: count 0) scaled.
hipError_t launch_grad_small(const GradSmall &g, const GradSmall &out, double *partial, float *norm, float max_norm,
                             float eps, hipStream_t stream);
hipError_t launch_grad_partials(const GradBatch &b, int32_t blocks, double *partial, hipStream_t stream);
// partial[0..n) summed into partial[0]; the norm to `norm` (fp32)
hipError_t launch_grad_total(double *partial, int32_t n, float *norm, hipStream_t stream);
// out = g * min(1, max_norm / (norm + eps)) from n partial sums; `norm` written when not null
hipError_t launch_grad_scale(const GradBatch &b, int32_t blocks, const double *partial, int32_t n, float *norm,
                             float max_norm, float eps, hipStream_t stream);

}  // namespace disco
