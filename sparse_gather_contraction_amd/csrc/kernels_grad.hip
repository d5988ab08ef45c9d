// kernels_grad.hip — the global norm of many gradients, and their scaling by min(1, max_norm / (norm + eps)).
//
// The tensors of a launch come in its arguments; a workgroup walks fixed chunks of them.  Squares are
// summed in fp64 (an fp32 gradient's square may leave fp32's range; at the memory's rate the fp64 adds cost
// nothing), each workgroup's sum goes to a place of its own, and the places are added in a fixed order, so
// the norm is bitwise reproducible.  Memory traffic bounds both passes: one read, then one read and one write.
#include "kernels.hpp"
#include "norm.hpp"
#include "norm_device.hpp"

namespace disco {

namespace {

constexpr int kThreads = 256;

// The last tensor whose first chunk is not past `id` (empty tensors have no chunks and share the next one's first).
__device__ __forceinline__ int find_tensor(const GradBatch &b, int id)
{
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.t[mid].first <= id) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ double sum_squares(const T *p, int n)
{
    constexpr int V = 16 / (int)sizeof(T), U = 4;
    const int t = threadIdx.x;
    double s0 = 0.0, s1 = 0.0;
    int i = t * V;
    for (; i + (U - 1) * kThreads * V + V <= n; i += U * kThreads * V) {
        Pack<T, V> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load_pack<T, V>(p + i + u * kThreads * V);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[V];
            unpack(r[u], f);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                s0 = __builtin_fma((double)f[e], (double)f[e], s0);
                s1 = __builtin_fma((double)f[e + 1], (double)f[e + 1], s1);
            }
        }
    }
    for (; i + V <= n; i += kThreads * V) {
        float f[V];
        load_f32<T, V>(p + i, f);
#pragma unroll
        for (int e = 0; e < V; ++e) s0 = __builtin_fma((double)f[e], (double)f[e], s0);
    }
    const int tail = n - n % V + t;
    if (tail < n) {
        const double f = load_elem(p, tail);
        s1 = __builtin_fma(f, f, s1);
    }
    return s0 + s1;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T *p, T *o, int n, float k)
{
    constexpr int V = 16 / (int)sizeof(T), U = 4;
    const int t = threadIdx.x;
    int i = t * V;
    for (; i + (U - 1) * kThreads * V + V <= n; i += U * kThreads * V) {
        Pack<T, V> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load_pack<T, V>(p + i + u * kThreads * V);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[V];
            unpack(r[u], f);
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] *= k;
            store_f32<T, V>(o + i + u * kThreads * V, f);
        }
    }
    for (; i + V <= n; i += kThreads * V) {
        float f[V];
        load_f32<T, V>(p + i, f);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] *= k;
        store_f32<T, V>(o + i, f);
    }
    const int tail = n - n % V + t;
    if (tail < n) store_elem(o, tail, load_elem(p, tail) * k);
}

// The sum of a value over the workgroup, the same in every thread.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double part[kThreads / 64];
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) v += part[i];
    return v;
}

__global__ __launch_bounds__(kThreads) void grad_partial_kernel(GradBatch b, double *partial)
{
    double s = 0.0;
    for (int id = blockIdx.x; id < b.chunks; id += gridDim.x) {
        const int i = find_tensor(b, id);
        const int64_t off = (int64_t)(id - b.t[i].first) * b.chunk, left = b.t[i].n - off;
        const int n = (int)(left < b.chunk ? left : b.chunk);
        const void *p = b.t[i].p;
        switch (b.t[i].dtype) {
        case 0: s += sum_squares((const float *)p + off, n); break;
        case 1: s += sum_squares((const bf16_t *)p + off, n); break;
        default: s += sum_squares((const f16_t *)p + off, n); break;
        }
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__device__ __forceinline__ double total_of(const double *partial, int n)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
    return block_sum(s);
}

__global__ __launch_bounds__(kThreads) void grad_total_kernel(double *partial, int n, float *norm)
{
    const double s = total_of(partial, n);
    if (threadIdx.x == 0) {
        if (n > 0) partial[0] = s;
        if (norm) *norm = (float)sqrt(s);
    }
}

// Chunks are walked from the last to the first: the ones that the sum read last are still in the caches.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradBatch b, const double *partial, int n, float *norm,
                                                              float max_norm, float eps)
{
    const double total = sqrt(total_of(partial, n));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    const double c = (double)max_norm / (total + (double)eps);
    const float k = (float)(c >= 1.0 ? 1.0 : c);  // a NaN norm gives NaN
    for (int id0 = blockIdx.x; id0 < b.chunks; id0 += gridDim.x) {
        const int id = b.chunks - 1 - id0, i = find_tensor(b, id);
        const int64_t off = (int64_t)(id - b.t[i].first) * b.chunk, left = b.t[i].n - off;
        const int len = (int)(left < b.chunk ? left : b.chunk);
        const void *p = b.t[i].p;
        void *o = b.t[i].o;
        if (p == o && k == 1.0f) continue;  // in place and unchanged
        switch (b.t[i].dtype) {
        case 0: scale_chunk((const float *)p + off, (float *)o + off, len, k); break;
        case 1: scale_chunk((const bf16_t *)p + off, (bf16_t *)o + off, len, k); break;
        default: scale_chunk((const f16_t *)p + off, (f16_t *)o + off, len, k); break;
        }
    }
}

}  // namespace

hipError_t launch_grad_partials(const GradBatch &b, int32_t blocks, double *partial, hipStream_t s)
{
    grad_partial_kernel<<<dim3(blocks), kThreads, 0, s>>>(b, partial);
    return hipGetLastError();
}

hipError_t launch_grad_total(double *partial, int32_t n, float *norm, hipStream_t s)
{
    grad_total_kernel<<<1, kThreads, 0, s>>>(partial, n, norm);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const GradBatch &b, int32_t blocks, const double *partial, int32_t n, float *norm,
                             float max_norm, float eps, hipStream_t s)
{
    grad_scale_kernel<<<dim3(blocks), kThreads, 0, s>>>(b, partial, n, norm, max_norm, eps);
    return hipGetLastError();
}

}  // namespace disco
