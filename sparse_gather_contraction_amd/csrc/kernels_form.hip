// kernels_form.hip — the 8-bit form of the channel products: its writer (with an activation function before it and a
// checkpoint of what the function was taken of) and its reader.
//
//   v = act(x);  scale = max(max |v| / 127, 2^-126) over a point's channels;  q = v / scale to whole numbers (ties to even)
//
// Everything between the load and q is fp32, the quotient by the scale as it is stored, so that q scale is the nearest
// such value to v.  Memory bounds the plain writer and the reader (2x256x721x1440 bf16: 300-316 and 343 us, 5.3 and 4.7 TB/s; rows
// of 2048 bf16 read back at 6.1), the vector units the writer with gelu and a checkpoint (259200x2048: 479-495 us; the function's
// exponential and reciprocal, and two quantisations of each value).  A point that holds a NaN or an infinity has scale NaN and
// q 0: what is computed from it is NaN.
#include "act_device.hpp"
#include "kernels.hpp"
#include "linear.hpp"
#include "norm_device.hpp"

namespace disco {

namespace {

constexpr int E = kFormChannels;

struct FormArgs {
    const void *x;
    void *out;
    int8_t *q, *kq;
    float *scale, *kscale;
    int64_t N, M;
    int32_t D, Dp, nv, lg, tiles_n;
    int32_t nt;        // stores past the caches
    FastDiv by_half;   // nv / 2 sixteens of a point
};

// A point's scale and its reciprocal in two parts, the first rounded correctly but for rare ties.  A quotient is the product with
// both, v inv + v low, off by 2^-46 before its one rounding (2^-28 for scales above 2^100, whose second part is subnormal).
struct I8Scale {
    float scale, inv, low;
};

__device__ __forceinline__ I8Scale i8_scale(float amax)
{
    if (!(amax < __builtin_inff())) return {__builtin_nanf(""), 0.0f, 0.0f};
    const float s = __builtin_fmaxf(amax / 127.0f, 0x1p-126f), r = __builtin_amdgcn_rcpf(s);
    const float inv = __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
    return {s, inv, __builtin_fmaf(-s, inv, 1.0f) * inv};
}

// Eight values to whole numbers in a byte each: the fp32 quotient by the scale as it is stored.  Added to 1.5 2^23 it is rounded
// to a whole number (ties to even) whose two's complement is the sum's low bits; |v / scale| <= 127 (1 + 2^-22), so none
// leaves a byte.
__device__ __forceinline__ u32x2 i8_codes(const float (&v)[E], const I8Scale &s)
{
    uint32_t b[E];
#pragma unroll
    for (int i = 0; i < E; ++i) b[i] = __float_as_uint(__builtin_fmaf(v[i], s.inv, v[i] * s.low) + 12582912.0f);
    u32x2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x0c0c0400u);
        r[i] = s.inv == 0.0f ? 0u : lo | hi << 16;  // NaN and infinite rows
    }
    return r;
}

__device__ __forceinline__ float amax_of(const float (&v)[E])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i += 2) m = max_abs(m, v[i], v[i + 1]);
    return m;
}

// Channels c .. c + 7 of a row, zeros from D on.
template <typename T>
__device__ __forceinline__ Pack<T, E> load_eight(const T *row, int c, int D)
{
    if (c + E <= D) return load_pack<T, E>(row + c);
    Pack<T, E> r;
#pragma unroll
    for (int i = 0; i < Pack<T, E>::kWords; ++i) {
        if constexpr (sizeof(T) == 4) {
            r.w[i] = c + i < D ? __float_as_uint(load_elem(row, c + i)) : 0u;
        } else {
            const uint16_t *p = (const uint16_t *)row;
            const uint32_t lo = c + 2 * i < D ? p[c + 2 * i] : 0u, hi = c + 2 * i + 1 < D ? p[c + 2 * i + 1] : 0u;
            r.w[i] = lo | hi << 16;
        }
    }
    return r;
}

// ---------------------------------------------------------------- rows (M = 1)

// The larger of a value over the 2^lg threads of a row: within a wave, then through LDS (one slot a wave).
__device__ __forceinline__ float row_max(float v, int lg, float *slots)
{
    v = join_run(v, lg, MaxOp());
    if (lg > 6) {
        const int wave = threadIdx.x >> 6, per_row = 1 << (lg - 6), first = wave & ~(per_row - 1);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) slots[wave] = v;
        __syncthreads();
        v = slots[first];
        for (int i = 1; i < per_row; ++i) v = MaxOp()(v, slots[first + i]);
    }
    return v;
}

template <typename T, int ACT, int KPT>
__global__ __launch_bounds__(kNormMaxThreads) void quantize_rows_kernel(FormArgs a)
{
    __shared__ float slots[2][kNormMaxThreads / 64];
    const int t = threadIdx.x, lanes = 1 << a.lg, tt = t & (lanes - 1);
    const int64_t want = (int64_t)blockIdx.x * (blockDim.x >> a.lg) + (t >> a.lg);
    const int64_t row = want < a.N ? want : a.N - 1;  // a slot past the end repeats the last row
    const T *x = (const T *)a.x + row * a.D;
    Pack<T, E> px[KPT];
#pragma unroll
    for (int k = 0; k < KPT; ++k) px[k] = load_eight(x, (k * lanes + tt) * E, a.D);
    float v[KPT][E], m = 0.0f, mk = 0.0f;
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        unpack(px[k], v[k]);
        if constexpr (ACT != DISCO_ACT_NONE) {
            mk = MaxOp()(mk, amax_of(v[k]));
#pragma unroll
            for (int i = 0; i < E; ++i) v[k][i] = act_value<ACT>(v[k][i]);
        }
        m = MaxOp()(m, amax_of(v[k]));
    }
    auto write = [&](float amax, int8_t *q, float *scale) {
        const I8Scale s = i8_scale(amax);
        q += row * a.Dp;
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            const int c = (k * lanes + tt) * E;
            const u32x2 w = i8_codes(v[k], s);
            if (c < a.Dp) {
                if (a.nt) store_as<true>(q + c, w);
                else store_as<false>(q + c, w);
            }
        }
        if (tt == 0) scale[row] = s.scale;
    };
    write(row_max(m, a.lg, slots[0]), a.q, a.scale);
    if constexpr (ACT != DISCO_ACT_NONE)
        if (a.kq) {
#pragma unroll
            for (int k = 0; k < KPT; ++k) unpack(px[k], v[k]);
            write(row_max(mk, a.lg, slots[1]), a.kq, a.kscale);
        }
}

// ---------------------------------------------------------------- fields

// A workgroup: 2^lg lanes along the points, nv threads along the channels.  LDS: [P][Dp] codes, [2][P] maxima.
template <typename T, int ACT, int VEC, int TH>
__global__ __launch_bounds__(TH) void quantize_field_kernel(FormArgs a)
{
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int t = threadIdx.x, lane = t & ((1 << a.lg) - 1), g = t >> a.lg, P = VEC << a.lg;
    const bool holds = g < a.nv;
    uint32_t *mx = (uint32_t *)(lds + (size_t)P * a.Dp);
    const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const ColPos pos = col_pos(tile, lane, VEC, a.lg, a.tiles_n, a.N, a.M);
    const T *x = (const T *)a.x + pos.n * a.D * a.M + pos.m;
    for (int i = t; i < 2 * P; i += blockDim.x) mx[i] = 0;
    Pack<T, VEC> px[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const int c = g * E + j;
        px[j] = load_pack<T, VEC>(x + (int64_t)(c < a.D ? c : a.D - 1) * a.M);
    }
    float v[E][VEC];
    auto take = [&](bool act, uint32_t *m) {
        float am[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) am[e] = 0.0f;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            unpack(px[j], v[j]);
            if (g * E + j >= a.D)  // the places behind D
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] = 0.0f;
            if constexpr (ACT != DISCO_ACT_NONE)
                if (act)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[j][e] = act_value<ACT>(v[j][e]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) am[e] = MaxOp()(am[e], __builtin_fabsf(v[j][e]));
        }
        if (holds)
#pragma unroll
            for (int e = 0; e < VEC; ++e) atomicMax(&m[lane * VEC + e], __float_as_uint(am[e]));
    };
    const int turn = lane % a.nv;
    int cg = g + turn;
    if (cg >= a.nv) cg -= a.nv;
    auto write = [&](const uint32_t *m, int8_t *q, float *scale) {
        // four points' scales at a time: all eight take registers that the values need (360x720 points of 2048 channels with gelu, a
        // checkpoint and two readers: 2097 us with eight, 1920 with four)
        constexpr int SP = VEC < 4 ? VEC : 4;
        if (holds)
#pragma unroll
            for (int e0 = 0; e0 < VEC; e0 += SP) {
                I8Scale s[SP];
#pragma unroll
                for (int e = 0; e < SP; ++e) s[e] = i8_scale(__uint_as_float(m[lane * VEC + e0 + e]));
                if (g == 0) {
                    float f[SP];
#pragma unroll
                    for (int e = 0; e < SP; ++e) f[e] = s[e].scale;
                    store_f32<float, SP>(scale + pos.n * a.M + pos.m + e0, f);
                }
#pragma unroll
                for (int e = 0; e < SP; ++e) {
                    float w[E];
#pragma unroll
                    for (int j = 0; j < E; ++j) w[j] = v[j][e0 + e];
                    *(u32x2 *)(lds + ((lane * VEC + e0 + e) * a.nv + cg) * 8) = i8_codes(w, s[e]);
                }
            }
        __syncthreads();
        const int half = a.nv >> 1;  // sixteens of a point
        for (int i = t; i < P * half; i += blockDim.x) {
            const int p = (int)a.by_half.div(i), h = i - p * half, l = p / VEC;
            const ColPos at = col_pos(tile, l, VEC, a.lg, a.tiles_n, a.N, a.M);
            const u32x2 lo = *(const u32x2 *)(lds + form_lds(p, 2 * h, a.nv, l));
            const u32x2 hi = *(const u32x2 *)(lds + form_lds(p, 2 * h + 1, a.nv, l));
            const u32x4 w = {lo.x, lo.y, hi.x, hi.y};
            int8_t *to = q + (at.n * a.M + at.m + (p - l * VEC)) * a.Dp + 16 * h;
            if (a.nt) store_as<true>(to, w);
            else store_as<false>(to, w);
        }
    };
    __syncthreads();
    take(true, mx);
    __syncthreads();
    write(mx, a.q, a.scale);
    if constexpr (ACT != DISCO_ACT_NONE)
        if (a.kq) {
            take(false, mx + P);
            __syncthreads();
            write(mx + P, a.kq, a.kscale);
        }
}

// ---------------------------------------------------------------- channels beyond the registers

// 2^lg lanes along the points, the threads walk the channels twice.
template <typename T, int ACT>
__global__ __launch_bounds__(kNormMaxThreads) void quantize_loop_kernel(FormArgs a)
{
    extern __shared__ uint32_t mxl[];
    const int t = threadIdx.x, P = 1 << a.lg, lane = t & (P - 1), g = t >> a.lg, groups = blockDim.x >> a.lg;
    const ColPos pos = col_pos(blockIdx.x, lane, 1, a.lg, 1, a.N, a.M);
    const T *x = (const T *)a.x + pos.n * a.D * a.M + pos.m;
    const int64_t point = pos.n * a.M + pos.m;
    for (int i = t; i < 2 * P; i += blockDim.x) mxl[i] = 0;
    __syncthreads();
    auto load = [&](int c, float (&v)[E]) {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = c + j < a.D ? load_elem(x, (int64_t)(c + j) * a.M) : 0.0f;
    };
    float m = 0.0f, mk = 0.0f;
    for (int c = g * E; c < a.D; c += groups * E) {
        float v[E];
        load(c, v);
        mk = MaxOp()(mk, amax_of(v));
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = act_value<ACT>(v[j]);
        m = MaxOp()(m, amax_of(v));
    }
    atomicMax(&mxl[lane], __float_as_uint(m));
    atomicMax(&mxl[P + lane], __float_as_uint(mk));
    __syncthreads();
    const I8Scale s = i8_scale(__uint_as_float(mxl[lane])), k = i8_scale(__uint_as_float(mxl[P + lane]));
    for (int c = g * E; c < a.Dp; c += groups * E) {
        float v[E], w[E];
        load(c, v);
#pragma unroll
        for (int j = 0; j < E; ++j) w[j] = act_value<ACT>(v[j]);
        *(u32x2 *)(a.q + point * a.Dp + c) = i8_codes(w, s);
        if (a.kq) *(u32x2 *)(a.kq + point * a.Dp + c) = i8_codes(v, k);
    }
    if (g == 0) {
        a.scale[point] = s.scale;
        if (a.kq) a.kscale[point] = k.scale;
    }
}

// ---------------------------------------------------------------- the reader

__device__ __forceinline__ void i8_values(u32x2 q, float scale, float (&f)[E])
{
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = (float)(int8_t)(q[i / 4] >> (8 * (i % 4))) * scale;
}

template <typename T>
__device__ __forceinline__ void store_eight(T *row, int c, int D, int nt, const float (&f)[E])
{
    if (c + E <= D) {
        if (nt) store_f32<T, E, true>(row + c, f);
        else store_f32<T, E>(row + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (c + i < D) store_elem(row, c + i, f[i]);
    }
}

template <typename T, int KPT>
__global__ __launch_bounds__(kNormMaxThreads) void dequantize_rows_kernel(FormArgs a)
{
    const int t = threadIdx.x, lanes = 1 << a.lg, tt = t & (lanes - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> a.lg) + (t >> a.lg);
    if (row >= a.N) return;
    const int8_t *q = a.q + row * a.Dp;
    const float scale = a.scale[row];
    u32x2 w[KPT];
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const int c = (k * lanes + tt) * E;
        w[k] = *(const u32x2 *)(q + (c < a.Dp ? c : 0));
    }
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        float f[E];
        i8_values(w[k], scale, f);
        store_eight((T *)a.out + row * a.D, (k * lanes + tt) * E, a.D, a.nt, f);
    }
}

template <typename T, int VEC, int TH>
__global__ __launch_bounds__(TH) void dequantize_field_kernel(FormArgs a)
{
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int t = threadIdx.x, lane = t & ((1 << a.lg) - 1), g = t >> a.lg, P = VEC << a.lg, half = a.nv >> 1;
    const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const ColPos pos = col_pos(tile, lane, VEC, a.lg, a.tiles_n, a.N, a.M);
    float s[VEC];
    load_f32<float, VEC>(a.scale + pos.n * a.M + pos.m, s);
    for (int i = t; i < P * half; i += blockDim.x) {
        const int p = (int)a.by_half.div(i), h = i - p * half, l = p / VEC;
        const ColPos at = col_pos(tile, l, VEC, a.lg, a.tiles_n, a.N, a.M);
        const u32x4 w = *(const u32x4 *)(a.q + (at.n * a.M + at.m + (p - l * VEC)) * a.Dp + 16 * h);
        const u32x2 lo = {w.x, w.y}, hi = {w.z, w.w};
        *(u32x2 *)(lds + form_lds(p, 2 * h, a.nv, l)) = lo;
        *(u32x2 *)(lds + form_lds(p, 2 * h + 1, a.nv, l)) = hi;
    }
    __syncthreads();
    if (g >= a.nv) return;
    float v[E][VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float f[E];
        i8_values(*(const u32x2 *)(lds + form_lds(lane * VEC + e, g, a.nv, lane)), s[e], f);
#pragma unroll
        for (int j = 0; j < E; ++j) v[j][e] = f[j];
    }
    T *out = (T *)a.out + pos.n * a.D * a.M + pos.m;
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (g * E + j < a.D) {
            T *to = out + (int64_t)(g * E + j) * a.M;
            if (a.nt) store_f32<T, VEC, true>(to, v[j]);
            else store_f32<T, VEC>(to, v[j]);
        }
}

template <typename T>
__global__ __launch_bounds__(kNormMaxThreads) void dequantize_loop_kernel(FormArgs a)
{
    const int t = threadIdx.x, lane = t & ((1 << a.lg) - 1), g = t >> a.lg, groups = blockDim.x >> a.lg;
    const ColPos pos = col_pos(blockIdx.x, lane, 1, a.lg, 1, a.N, a.M);
    T *out = (T *)a.out + pos.n * a.D * a.M + pos.m;
    const int64_t point = pos.n * a.M + pos.m;
    const float scale = a.scale[point];
    for (int c = g * E; c < a.D; c += groups * E) {
        float f[E];
        i8_values(*(const u32x2 *)(a.q + point * a.Dp + c), scale, f);
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (c + j < a.D) store_elem(out, (int64_t)(c + j) * a.M, f[j]);
    }
}

FormArgs form_args(const FormLaunch &l, const FormGeom &g)
{
    FormArgs a;
    a.x = l.x; a.out = l.out; a.q = l.q; a.kq = l.kq; a.scale = l.scale; a.kscale = l.kscale;
    a.N = l.N; a.M = l.M; a.D = (int32_t)l.D; a.Dp = (int32_t)padded_channels(l.D);
    a.nv = a.Dp / E; a.lg = g.lg; a.tiles_n = g.tiles_n;
    const int64_t P = l.N * l.M, esz = l.dtype == 0 ? 4 : 2;
    // (2x256x721x1440 bf16 there and back 661 -> 647 us, 80x721x1440 108 -> 101)
    a.nt = l.x ? stream_stores(true, P * a.Dp, a.Dp, l.q, l.kq)
               : stream_stores(l.M == 1, P * l.D * esz, (l.M == 1 ? l.D : l.M) * esz, l.out, nullptr);
    a.by_half = fast_div((uint32_t)a.nv / 2);
    return a;
}

// A field kernel's launch: 2048 channels of 32 points take a little more LDS than the 64 KiB that a kernel has without asking.
template <typename K>
hipError_t launch_field(K kernel, dim3 grid, dim3 block, size_t lds, hipStream_t s, const FormArgs &a)
{
    if (lds > (64u << 10)) {
        const hipError_t e = allow_lds((const void *)kernel, lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<grid, block, lds, s>>>(a);
    return hipGetLastError();
}

template <typename T, int ACT>
hipError_t quantize_act(const FormLaunch &l, hipStream_t s)
{
    const FormGeom g = form_geom(l.N, l.D, l.M, (int)sizeof(T));
    const FormArgs a = form_args(l, g);
    const dim3 grid((uint32_t)g.tiles), block(g.threads);
    const size_t lds = form_lds_bytes(g, a.Dp);
    constexpr int V = 16 / (int)sizeof(T);
    if (g.loop) quantize_loop_kernel<T, ACT><<<grid, block, lds, s>>>(a);
    else if (g.rows && g.per == 1) quantize_rows_kernel<T, ACT, 1><<<grid, block, 0, s>>>(a);
    else if (g.rows && g.per == 2) quantize_rows_kernel<T, ACT, 2><<<grid, block, 0, s>>>(a);
    else if (g.rows) quantize_rows_kernel<T, ACT, 4><<<grid, block, 0, s>>>(a);
    else if (g.vec > 1 && g.threads > kFormThreads) return launch_field(quantize_field_kernel<T, ACT, V, kNormMaxThreads>, grid, block, lds, s, a);
    else if (g.vec > 1) return launch_field(quantize_field_kernel<T, ACT, V, kFormThreads>, grid, block, lds, s, a);
    else return launch_field(quantize_field_kernel<T, ACT, 1, kNormMaxThreads>, grid, block, lds, s, a);
    return hipGetLastError();
}

template <typename T>
hipError_t quantize_typed(const FormLaunch &l, hipStream_t s)
{
    return l.act == DISCO_ACT_GELU ? quantize_act<T, DISCO_ACT_GELU>(l, s)
         : l.act == DISCO_ACT_SILU ? quantize_act<T, DISCO_ACT_SILU>(l, s)
                                   : quantize_act<T, DISCO_ACT_NONE>(l, s);
}

template <typename T>
hipError_t dequantize_typed(const FormLaunch &l, hipStream_t s)
{
    const FormGeom g = form_geom(l.N, l.D, l.M, (int)sizeof(T));
    const FormArgs a = form_args(l, g);
    const dim3 grid((uint32_t)g.tiles), block(g.threads);
    const size_t lds = form_lds_bytes(g, a.Dp);
    constexpr int V = 16 / (int)sizeof(T);
    if (g.loop) dequantize_loop_kernel<T><<<grid, block, 0, s>>>(a);
    else if (g.rows && g.per == 1) dequantize_rows_kernel<T, 1><<<grid, block, 0, s>>>(a);
    else if (g.rows && g.per == 2) dequantize_rows_kernel<T, 2><<<grid, block, 0, s>>>(a);
    else if (g.rows) dequantize_rows_kernel<T, 4><<<grid, block, 0, s>>>(a);
    else if (g.vec > 1) return launch_field(dequantize_field_kernel<T, V, kNormMaxThreads>, grid, block, lds, s, a);
    else return launch_field(dequantize_field_kernel<T, 1, kNormMaxThreads>, grid, block, lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_i8(const FormLaunch &l, hipStream_t s)
{
    return l.dtype == 0 ? quantize_typed<float>(l, s) : l.dtype == 1 ? quantize_typed<bf16_t>(l, s) : quantize_typed<f16_t>(l, s);
}

hipError_t launch_dequantize_i8(const FormLaunch &l, hipStream_t s)
{
    return l.dtype == 0 ? dequantize_typed<float>(l, s) : l.dtype == 1 ? dequantize_typed<bf16_t>(l, s) : dequantize_typed<f16_t>(l, s);
}

}  // namespace disco
