// kernels_grad.hip — the global norm of many gradients, and their scaling by min(1, max_norm / (norm + eps)).
//
// The tensors of a launch come in its arguments; a workgroup walks fixed chunks of them.  Squares are
// summed in fp64 (an fp32 gradient's square may leave fp32's range; at the memory's rate the fp64 adds cost
// nothing), each workgroup's sum goes to a place of its own, and the places are added in a fixed order, so
// the norm is bitwise reproducible.  Memory traffic bounds both passes: one read, then one read and one write.
// 2^28 fp32 elements: 153-168 us (6.4-7.0 TB/s) and 374-391 us (5.5-5.7 TB/s); 12.6 M bf16 elements, which fit the
// last-level cache: 7.4 and 12.8 us.
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

// Calls body(packs, at, full) for each run of kUnroll vectors that thread t of kThreads holds of p[0..n); `full`: all
// are whole vectors inside, else vector u is one only if at + u * kThreads * V + V <= n.
template <typename T, bool NT, typename F>
__device__ __forceinline__ void walk(const T *p, int n, int t, F body)
{
    constexpr int V = 16 / (int)sizeof(T), S = kThreads * V;
    for (int i0 = 0; i0 + V <= n; i0 += kUnroll * S) {
        const int i = i0 + t * V;
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
__device__ __forceinline__ double sum_squares(const T *p, int n, int t)
{
    constexpr int V = 16 / (int)sizeof(T), S = kThreads * V;
    double s0 = 0.0, s1 = 0.0;
    walk<T, NT>(p, n, t, [&](const Pack<T, V> (&r)[kUnroll], int i, bool full) {
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
    const int tail = n - n % V + t;
    if (tail < n) {
        const double f = load_elem(p, tail);
        s1 = __builtin_fma(f, f, s1);
    }
    return s0 + s1;
}

template <typename T, bool NT, typename K>
__device__ __forceinline__ void scale_by(const T *p, T *o, int n, K k, int t)
{
    constexpr int V = 16 / (int)sizeof(T), S = kThreads * V;
    walk<T, NT>(p, n, t, [&](const Pack<T, V> (&r)[kUnroll], int i, bool full) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (full || i + u * S + V <= n) {
                float f[V];
                unpack(r[u], f);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = (float)(f[e] * k);
                store_f32<T, V, NT>(o + i + u * S, f);
            }
    });
    const int tail = n - n % V + t;
    if (tail < n) store_elem(o, tail, (float)(load_elem(p, tail) * k));
}

// The factor of the gradients, in fp32 and, where it lies below fp32's normal range, as it was computed: a subnormal
// fp32 factor has few bits or none left where the products have all of theirs (gradients of 1e38 by 1e-43).
struct Factor {
    float k;
    double c;   // 0: k is all there is to it
};

template <typename T, bool NT>
__device__ __forceinline__ void scale_chunk(const T *p, T *o, int n, const Factor &k, int t)
{
    if (k.c == 0.0) scale_by<T, NT>(p, o, n, k.k, t);
    else scale_by<T, false>(p, o, n, k.c, t);
}

// The sum of a value over the workgroup of THREADS, the same in every thread.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double part[THREADS / 64];
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) v += part[i];
    return v;
}

template <typename T>
__device__ __forceinline__ double sum_tensor(const GradTensor &t, int64_t off, int n, bool nt)
{
    const T *p = (const T *)t.p + off;
    return nt ? sum_squares<T, true>(p, n, threadIdx.x) : sum_squares<T, false>(p, n, threadIdx.x);
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
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__device__ __forceinline__ double total_of(const double *partial, int n)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
    return block_sum<kThreads>(s);
}

__global__ __launch_bounds__(kThreads) void grad_total_kernel(double *partial, int n, float *norm)
{
    const double s = total_of(partial, n);
    if (threadIdx.x == 0) {
        partial[0] = s;
        if (norm) *norm = (float)sqrt(s);
    }
}

template <typename T>
__device__ __forceinline__ void scale_tensor(const GradTensor &t, int64_t off, int n, const Factor &k, bool nt)
{
    const T *p = (const T *)t.p + off;
    T *o = (T *)t.o + off;
    if (nt) scale_chunk<T, true>(p, o, n, k, threadIdx.x);
    else scale_chunk<T, false>(p, o, n, k, threadIdx.x);
}

// The factor of a total norm: min(1, max_norm / (total + eps)), 1 where both are 0 (nothing to clip) and 0 for an
// infinite norm whatever max_norm is; a NaN norm gives NaN.
__device__ __forceinline__ Factor clip_factor(double total, float max_norm, float eps)
{
    const double t = total + (double)eps;
    if (__builtin_isinf(t)) return {0.0f, 0.0};
    if ((double)max_norm >= t) return {1.0f, 0.0};
    const double c = (double)max_norm / t;
    return {(float)c, c < 0x1p-126 ? c : 0.0};
}

// Few elements: one workgroup sums all chunks and scales them, kThreads threads a chunk.
__global__ __launch_bounds__(1024) void grad_small_kernel(GradSmall g, GradSmall out, double *partial, float *norm,
                                                          float max_norm, float eps)
{
    const int first = threadIdx.x / kThreads, t = threadIdx.x % kThreads, step = 1024 / kThreads;
    double s = 0.0;
    for (int i = first; i < g.count; i += step) {
        const GradTensor &v = g.t[i];
        switch (v.dtype) {
        case 0: s += sum_squares<float, false>((const float *)v.p, (int)v.n, t); break;
        case 1: s += sum_squares<bf16_t, false>((const bf16_t *)v.p, (int)v.n, t); break;
        default: s += sum_squares<f16_t, false>((const f16_t *)v.p, (int)v.n, t); break;
        }
    }
    s = block_sum<1024>(s);
    const double total = sqrt(s);
    if (threadIdx.x == 0) {
        partial[0] = s;
        *norm = (float)total;
    }
    const Factor k = clip_factor(total, max_norm, eps);
    for (int i = first; i < out.count; i += step) {
        const GradTensor &v = out.t[i];
        if (v.p == v.o && k.k == 1.0f) continue;  // in place and unchanged
        switch (v.dtype) {
        case 0: scale_chunk<float, false>((const float *)v.p, (float *)v.o, (int)v.n, k, t); break;
        case 1: scale_chunk<bf16_t, false>((const bf16_t *)v.p, (bf16_t *)v.o, (int)v.n, k, t); break;
        default: scale_chunk<f16_t, false>((const f16_t *)v.p, (f16_t *)v.o, (int)v.n, k, t); break;
        }
    }
}

// Chunks are walked from the last to the first: the ones that the sum read last are still in the caches.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradBatch b, const double *partial, int n, float *norm,
                                                              float max_norm, float eps)
{
    const Firsts firsts = load_firsts(b);
    const double total = sqrt(total_of(partial, n));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    const Factor k = clip_factor(total, max_norm, eps);
    for (int id0 = blockIdx.x; id0 < b.chunks; id0 += gridDim.x) {
        const int id = b.chunks - 1 - id0;
        const GradTensor &t = b.t[find_tensor(firsts, id)];
        const int64_t off = (int64_t)(id - t.first) * b.chunk, left = t.n - off;
        const int len = (int)(left < b.chunk ? left : b.chunk);
        if (t.p == t.o && k.k == 1.0f) continue;  // in place and unchanged
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

hipError_t launch_grad_small(const GradSmall &g, const GradSmall &out, double *partial, float *norm, float max_norm,
                             float eps, hipStream_t s)
{
    grad_small_kernel<<<1, 1024, 0, s>>>(g, out, partial, norm, max_norm, eps);
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
