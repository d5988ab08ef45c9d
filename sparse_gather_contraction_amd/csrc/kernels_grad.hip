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
constexpr int kUnroll = 4;   // vectors that a thread has in flight

// The tensors' first chunks, held over the lanes of each wave: two a lane.
struct Firsts {
    int32_t lo, hi;
};

__device__ __forceinline__ Firsts load_firsts(const GradBatch &b)
{
    const int l = threadIdx.x & 63;
    Firsts f;
    f.lo = l < b.count ? b.t[l].first : INT32_MAX;
    f.hi = l + 64 < b.count ? b.t[l + 64].first : INT32_MAX;
    return f;
}

// The tensor of chunk `id`: the last one whose first chunk is not past it.
__device__ __forceinline__ int find_tensor(const Firsts &f, int id)
{
    return __popcll(__ballot(f.lo <= id)) + __popcll(__ballot(f.hi <= id)) - 1;
}

// Calls body(packs, at, full) for each run of kUnroll vectors a thread holds of p[0..n); `full`: all are whole
// vectors inside, else vector u is one only if at + u * kThreads * V + V <= n.
template <typename T, bool NT, typename F>
__device__ __forceinline__ void walk(const T *p, int n, F body)
{
    constexpr int V = 16 / (int)sizeof(T), S = kThreads * V;
    for (int i0 = 0; i0 + V <= n; i0 += kUnroll * S) {
        const int i = i0 + (int)threadIdx.x * V;
        Pack<T, V> r[kUnroll];
        if (i0 + kUnroll * S <= n) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) r[u] = load_pack<T, V, NT>(p + i + u * S);
            body(r, i, true);
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (i + u * S + V <= n) r[u] = load_pack<T, V, NT>(p + i + u * S);
            body(r, i, false);
        }
    }
}

template <typename T, bool NT>
__device__ __forceinline__ double sum_squares(const T *p, int n)
{
    constexpr int V = 16 / (int)sizeof(T), S = kThreads * V;
    double s0 = 0.0, s1 = 0.0;
    walk<T, NT>(p, n, [&](const Pack<T, V> (&r)[kUnroll], int i, bool full) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (full || i + u * S + V <= n) {
                float f[V];
                unpack(r[u], f);
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    s0 = __builtin_fma((double)f[e], (double)f[e], s0);
                    s1 = __builtin_fma((double)f[e + 1], (double)f[e + 1], s1);
                }
            }
    });
    const int tail = n - n % V + (int)threadIdx.x;
    if (tail < n) {
        const double f = load_elem(p, tail);
        s1 = __builtin_fma(f, f, s1);
    }
    return s0 + s1;
}

template <typename T, bool NT>
__device__ __forceinline__ void scale_chunk(const T *p, T *o, int n, float k)
{
    constexpr int V = 16 / (int)sizeof(T), S = kThreads * V;
    walk<T, NT>(p, n, [&](const Pack<T, V> (&r)[kUnroll], int i, bool full) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (full || i + u * S + V <= n) {
                float f[V];
                unpack(r[u], f);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] *= k;
                store_f32<T, V, NT>(o + i + u * S, f);
            }
    });
    const int tail = n - n % V + (int)threadIdx.x;
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

template <typename T>
__device__ __forceinline__ double sum_tensor(const GradTensor &t, int64_t off, int n, bool nt)
{
    const T *p = (const T *)t.p + off;
    return nt ? sum_squares<T, true>(p, n) : sum_squares<T, false>(p, n);
}

__global__ __launch_bounds__(kThreads) void grad_partial_kernel(GradBatch b, double *partial)
{
    const Firsts firsts = load_firsts(b);
    double s = 0.0;
    for (int id = blockIdx.x; id < b.chunks; id += gridDim.x) {
        const GradTensor &t = b.t[find_tensor(firsts, id)];
        const int64_t off = (int64_t)(id - t.first) * b.chunk, left = t.n - off;
        const int n = (int)(left < b.chunk ? left : b.chunk);
        switch (t.dtype) {
        case 0: s += sum_tensor<float>(t, off, n, b.stream); break;
        case 1: s += sum_tensor<bf16_t>(t, off, n, b.stream); break;
        default: s += sum_tensor<f16_t>(t, off, n, b.stream); break;
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

template <typename T>
__device__ __forceinline__ void scale_tensor(const GradTensor &t, int64_t off, int n, float k, bool nt)
{
    const T *p = (const T *)t.p + off;
    T *o = (T *)t.o + off;
    if (nt) scale_chunk<T, true>(p, o, n, k);
    else scale_chunk<T, false>(p, o, n, k);
}

// Chunks are walked from the last to the first: the ones that the sum read last are still in the caches.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradBatch b, const double *partial, int n, float *norm,
                                                              float max_norm, float eps)
{
    const Firsts firsts = load_firsts(b);
    const double total = sqrt(total_of(partial, n));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    const double c = (double)max_norm / (total + (double)eps);
    const float k = (float)(c >= 1.0 ? 1.0 : c);  // a NaN norm gives NaN
    for (int id0 = blockIdx.x; id0 < b.chunks; id0 += gridDim.x) {
        const int id = b.chunks - 1 - id0;
        const GradTensor &t = b.t[find_tensor(firsts, id)];
        const int64_t off = (int64_t)(id - t.first) * b.chunk, left = t.n - off;
        const int len = (int)(left < b.chunk ? left : b.chunk);
        if (t.p == t.o && k == 1.0f) continue;  // in place and unchanged
        switch (t.dtype) {
        case 0: scale_tensor<float>(t, off, len, k, b.stream); break;
        case 1: scale_tensor<bf16_t>(t, off, len, k, b.stream); break;
        default: scale_tensor<f16_t>(t, off, len, k, b.stream); break;
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
