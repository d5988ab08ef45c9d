// norm_device.hpp — vector loads, stores and conversions of the norm, 8-bit and gradient kernels.
#pragma once

#include "common.hpp"

namespace disco {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// VEC elements of T as they lie in memory.  Loads and stores need the element's alignment only.
template <typename T, int VEC>
struct Pack {
    static constexpr int kBytes = VEC * (int)sizeof(T);
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];
};

// A load that the caches keep, or (NT) one that is dropped by them first.
template <bool NT, typename V, typename T>
__device__ __forceinline__ V load_as(const T *p)
{
    V v;
    if constexpr (NT) {
        typedef V VU __attribute__((aligned(1)));
        v = __builtin_nontemporal_load((const VU *)p);
    } else {
        __builtin_memcpy(&v, p, sizeof(V));
    }
    return v;
}

template <typename T, int VEC, bool NT = false>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p)
{
    constexpr int B = Pack<T, VEC>::kBytes;
    Pack<T, VEC> r;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
            const u32x4 v = load_as<NT, u32x4>(p + i * (16 / (int)sizeof(T)));
            r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (B == 8) {
        const u32x2 v = load_as<NT, u32x2>(p);
        r.w[0] = v.x; r.w[1] = v.y;
    } else if constexpr (B == 4) {
        r.w[0] = load_as<NT, uint32_t>(p);
    } else if constexpr (B == 2) {
        r.w[0] = *(const uint16_t *)p;
    } else {
        static_assert(B == 1, "pack size");
        r.w[0] = *(const uint8_t *)p;
    }
    return r;
}

// A store that the caches keep, or (NT) one that passes through them.
template <bool NT, typename V, typename T>
__device__ __forceinline__ void store_as(T *p, const V &v)
{
    if constexpr (NT) {
        typedef V VU __attribute__((aligned(1)));
        __builtin_nontemporal_store(v, (VU *)p);
    } else {
        __builtin_memcpy(p, &v, sizeof(V));
    }
}

template <typename T, int VEC, bool NT = false>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &r)
{
    constexpr int B = Pack<T, VEC>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
            const u32x4 v = {r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
            store_as<NT>(p + i * (16 / (int)sizeof(T)), v);
        }
    } else if constexpr (B == 8) {
        const u32x2 v = {r.w[0], r.w[1]};
        store_as<NT>(p, v);
    } else if constexpr (B == 4) {
        store_as<NT>(p, r.w[0]);
    } else if constexpr (B == 2) {
        *(uint16_t *)p = (uint16_t)r.w[0];
    } else {
        *(uint8_t *)p = (uint8_t)r.w[0];
    }
}

// Keeps the values as they lie, in their registers: what is unpacked after this is not the fp32 values
// unpacked before it, which would hold twice the registers of 16-bit elements.
template <typename T, int VEC>
__device__ __forceinline__ void keep_packed(Pack<T, VEC> &r)
{
    if constexpr (sizeof(T) == 2 && VEC > 1)
#pragma unroll
        for (int i = 0; i < Pack<T, VEC>::kWords; ++i) asm volatile("" : "+v"(r.w[i]));
}

// The values are made here and not put off until they are used.
__device__ __forceinline__ void keep_here(float &v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void keep_here(double &v) { asm volatile("" : "+v"(v)); }

template <typename T, int VEC>
__device__ __forceinline__ void keep_here(Pack<T, VEC> &r)
{
#pragma unroll
    for (int i = 0; i < Pack<T, VEC>::kWords; ++i) asm volatile("" : "+v"(r.w[i]));
}

template <int VEC>
__device__ __forceinline__ void unpack(const Pack<float, VEC> &r, float (&f)[VEC])
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(r.w[i]);
}

template <int VEC>
__device__ __forceinline__ void unpack(const Pack<bf16_t, VEC> &r, float (&f)[VEC])
{
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        f[i] = __uint_as_float((i & 1) ? (r.w[i / 2] & 0xffff0000u) : (r.w[i / 2] << 16));
}

template <int VEC>
__device__ __forceinline__ void unpack(const Pack<f16_t, VEC> &r, float (&f)[VEC])
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const f16x2 h = __builtin_bit_cast(f16x2, r.w[i / 2]);
        f[i] = (float)((i & 1) ? h.y : h.x);
    }
}

// fp32 -> the element type, each value rounded once (round to nearest even)
template <int VEC>
__device__ __forceinline__ void pack(const float (&f)[VEC], Pack<float, VEC> &r)
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.w[i] = __float_as_uint(f[i]);
}

template <int VEC>
__device__ __forceinline__ void pack(const float (&f)[VEC], Pack<bf16_t, VEC> &r)
{
    if constexpr (VEC == 1) {
        r.w[0] = f32_to_bf16(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const f32x2 v = {f[2 * i], f[2 * i + 1]};
            r.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
        }
    }
}

template <int VEC>
__device__ __forceinline__ void pack(const float (&f)[VEC], Pack<f16_t, VEC> &r)
{
    if constexpr (VEC == 1) {
        r.w[0] = __builtin_bit_cast(uint16_t, (f16_t)f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const f32x2 v = {f[2 * i], f[2 * i + 1]};
            r.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_f32(const T *p, float (&f)[VEC])
{
    unpack(load_pack<T, VEC>(p), f);
}

template <typename T, int VEC, bool NT = false>
__device__ __forceinline__ void store_f32(T *p, const float (&f)[VEC])
{
    Pack<T, VEC> r;
    pack(f, r);
    store_pack<T, VEC, NT>(p, r);
}

// 8-bit values (fmt 0: e4m3, 1: e5m2, both with the OCP encodings gfx950 converts to), round to nearest even
template <int VEC>
__device__ __forceinline__ void pack_f8(const float (&f)[VEC], int fmt, Pack<uint8_t, VEC> &r)
{
    if constexpr (VEC == 1) {
        const int v = fmt ? __builtin_amdgcn_cvt_pk_bf8_f32(f[0], 0.0f, 0, false)
                          : __builtin_amdgcn_cvt_pk_fp8_f32(f[0], 0.0f, 0, false);
        r.w[0] = (uint32_t)v & 0xffu;
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            int v = 0;
            if (fmt) {
                v = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i], f[4 * i + 1], v, false);
                v = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i + 2], f[4 * i + 3], v, true);
            } else {
                v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], v, false);
                v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], v, true);
            }
            r.w[i] = (uint32_t)v;
        }
    }
}

template <int VEC>
__device__ __forceinline__ void unpack_f8(const Pack<uint8_t, VEC> &r, int fmt, float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        const f32x2 v = fmt ? __builtin_amdgcn_cvt_pk_f32_bf8((int)r.w[0], false)
                            : __builtin_amdgcn_cvt_pk_f32_fp8((int)r.w[0], false);
        f[0] = v.x;
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const f32x2 a = fmt ? __builtin_amdgcn_cvt_pk_f32_bf8((int)r.w[i], false)
                                : __builtin_amdgcn_cvt_pk_f32_fp8((int)r.w[i], false);
            const f32x2 b = fmt ? __builtin_amdgcn_cvt_pk_f32_bf8((int)r.w[i], true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8((int)r.w[i], true);
            f[4 * i] = a.x; f[4 * i + 1] = a.y; f[4 * i + 2] = b.x; f[4 * i + 3] = b.y;
        }
    }
}

// The norm's weight, fp32 or of the data type.
template <typename T>
__device__ __forceinline__ float load_weight(const void *w, int wf32, int64_t c)
{
    return wf32 ? ((const float *)w)[c] : load_elem((const T *)w, c);
}

// |v| as an unsigned whole number: ordered like the values, with infinity and then NaN above them
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// max(m, |a|, |b|), a NaN kept
__device__ __forceinline__ float max_abs(float m, float a, float b)
{
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(a)), __builtin_fabsf(b));
}

// ---- joins over the lanes of a wave: DPP moves and the row and half swaps, which need no LDS

struct AddOp {
    template <typename V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct MaxOp {  // of values that are 0 or more; a NaN is kept
    __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_elementwise_maximum(a, b); }
};

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}

template <int CTRL>
__device__ __forceinline__ double dpp(double v)
{
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    const u32x2 r = {(uint32_t)__builtin_amdgcn_mov_dpp((int)w.x, CTRL, 0xf, 0xf, true),
                     (uint32_t)__builtin_amdgcn_mov_dpp((int)w.y, CTRL, 0xf, 0xf, true)};
    return __builtin_bit_cast(double, r);
}

// v of the lane's row of 16 and of the row beside it (lane ^ 16), in an order that both rows share
template <typename Op>
__device__ __forceinline__ float join16(float v, Op op)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <typename Op>
__device__ __forceinline__ double join16(double v, Op op)
{
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    const auto x = __builtin_amdgcn_permlane16_swap(w.x, w.x, false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(w.y, w.y, false, false);
    const u32x2 a = {x[0], y[0]}, b = {x[1], y[1]};
    return op(__builtin_bit_cast(double, a), __builtin_bit_cast(double, b));
}

// the same over the wave's halves (lane ^ 32)
template <typename Op>
__device__ __forceinline__ float join32(float v, Op op)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <typename Op>
__device__ __forceinline__ double join32(double v, Op op)
{
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    const auto x = __builtin_amdgcn_permlane32_swap(w.x, w.x, false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(w.y, w.y, false, false);
    const u32x2 a = {x[0], y[0]}, b = {x[1], y[1]};
    return op(__builtin_bit_cast(double, a), __builtin_bit_cast(double, b));
}

// Joins v over each run of 2^lg lanes (lg <= 6, uniform), every lane of a run getting the same value.
template <typename V, typename Op>
__device__ __forceinline__ V join_run(V v, int lg, Op op)
{
    if (lg > 0) v = op(v, dpp<0xB1>(v));   // quad_perm 1 0 3 2
    if (lg > 1) v = op(v, dpp<0x4E>(v));   // quad_perm 2 3 0 1
    if (lg > 2) v = op(v, dpp<0x141>(v));  // half mirror: the other quad of the eight, whose lanes agree by now
    if (lg > 3) v = op(v, dpp<0x140>(v));  // mirror: the other eight of the row
    if (lg > 4) v = join16(v, op);
    if (lg > 5) v = join32(v, op);
    return v;
}

// Joins v over the lanes of a wave that are 2^lg apart.
template <typename Op>
__device__ __forceinline__ float join_apart(float v, int lg, Op op)
{
    for (int o = lg; o < 4; ++o) v = op(v, __shfl_xor(v, 1 << o));
    if (lg < 5) v = join16(v, op);
    if (lg < 6) v = join32(v, op);
    return v;
}

// The scale of a group whose largest |y| is amax (0 or more) and what takes its values to their quotients.
//   scale = amax / qmax, at least 2^-126 (the reciprocal of a smaller one leaves fp32's range).
// A quotient is y / scale by the scale as it is stored, which the reader multiplies by: the product with the
// reciprocal (off by 2^-23 at most), then its remainder y - q scale brought in, two fma an element.  That is off by
// 2^-45 before its one rounding to fp32; the product alone, off by the reciprocal's error too, sent values next to
// a tie to the other code.
// amax infinite: scale infinite, a finite y gives 0 and an infinite one NaN (inv and back are 0: with the
// infinite scale itself the remainder of a finite y would be NaN); amax NaN: all NaN.
struct F8Scale {
    float scale, inv, back;
};

__device__ __forceinline__ F8Scale f8_scale(float amax, float qmax)
{
    // amax / qmax by the product with the rounded 1 / qmax and its remainder: for these two qmax the same fp32 number as
    // division gives, for every finite amax whose scale is 2^-126 or more (all of them tried), in a third of its steps
    // (259200x512 fp16 72.3 against 75.6 us)
    const float r = qmax == 448.0f ? 1.0f / 448.0f : 1.0f / 57344.0f, q = amax * r;
    const float s = amax < __builtin_inff() ? __builtin_fmaf(__builtin_fmaf(-q, qmax, amax), r, q) : amax;
    if (s < 0x1p-126f) return {0x1p-126f, 0x1p126f, 0x1p-126f};
    const float inv = __builtin_amdgcn_rcpf(s);
    return {s, inv, inv == 0.0f ? 0.0f : s};
}

__device__ __forceinline__ float f8_quot(float y, float inv, float back)
{
    const float q = y * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, back, y), inv, q);
}

}  // namespace disco
