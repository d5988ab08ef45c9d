// linear_device.hpp — what the tiles of the channel products share on the device: direct loads, the points of a
// field, and the way of an output tile from the matrix cores' accumulators to memory.
#pragma once

#include "linear_plan.hpp"
#include "norm_device.hpp"

namespace disco {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef void __attribute__((address_space(3))) *lds_ptr_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t lin_rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)bytes, 0x00020000);
}

// Lane i of the instruction writes LDS base `l` + 16 i.
__device__ __forceinline__ void lin_dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, void *l)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)l, 16, voff, 0, 0, 0);
}

// The same, and one of 4 bytes, as instructions whose landing the kernel waits for itself (wait_vm): the compiler puts a wait
// for every direct load in flight before an LDS read of another array.  They write m0 and no other register (a kernel that
// uses them has no other use for m0, which the compiler sets before each of its own); `l` and the descriptor are
// uniform; the waits cover a descriptor or m0 written just before.
typedef uint32_t rsrc4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ rsrc4_t lin_rsrc4(const void *base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)base;
    return {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b), (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xffffu)),
            (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

__device__ __forceinline__ uint32_t lds_offset(const void *l) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_ptr_t)l); }

__device__ __forceinline__ void lin_dma16_free(rsrc4_t r, uint32_t voff, uint32_t l)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "s"(l), "v"(voff), "s"(r) : "memory");
}

__device__ __forceinline__ void lin_dma4_free(rsrc4_t r, uint32_t voff, uint32_t l)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "s"(l), "v"(voff), "s"(r) : "memory");
}

constexpr uint32_t kLinOob = 0x80000000u;  // beyond every buffer used here: the load gives zeros

// Waits until at most N of this wave's memory operations are in flight, and for all its LDS operations.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N < 64, "a count of six bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4 << 14));
}

// A barrier of the workgroup that leaves direct loads in flight (__syncthreads() waits for them all); LDS accesses stay on
// their side of it.
__device__ __forceinline__ void bare_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A tensor with one axis that lies together (c) and one that does not (j): element (j, c) lies at run(c) + j stride().
// PLANES: c are points in planes of M with J channels; else rows of ld.
struct Planes {
    FastDiv by_m;
    int64_t M, J, ld;
    template <bool PLANES>
    __device__ __forceinline__ int64_t run(uint32_t c) const
    {
        if (!PLANES) return c;
        const uint32_t n = by_m.div(c);
        return (int64_t)n * (J - 1) * M + c;   // n J M + (c - n M)
    }
    template <bool PLANES>
    __device__ __forceinline__ int64_t stride() const { return PLANES ? M : ld; }
    // whether c .. c + 7 lie together below len
    template <bool PLANES>
    __device__ __forceinline__ bool whole(uint32_t c, uint32_t len) const
    {
        return c + 8 <= len && (!PLANES || c - by_m.div(c) * (uint32_t)M + 8 <= (uint32_t)M);
    }
};

// Eight 16-bit elements (j, c .. c + 7), zeros where c passes len.  Rows j are the caller's to bound.
template <bool PLANES>
__device__ __forceinline__ u32x4 load_run(const uint16_t *base, const Planes &pl, int64_t j, uint32_t c, uint32_t len)
{
    const uint16_t *row = base + j * pl.stride<PLANES>();
    if (pl.whole<PLANES>(c, len)) return load_as<false, u32x4>(row + pl.run<PLANES>(c));
    u32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < len) r[i / 2] |= (uint32_t)row[pl.run<PLANES>(c + i)] << (16 * (i & 1));
    return r;
}

// One lane's 16-byte pieces of an output whose axis u lies together: the places (v, u .. u + n-1), n = 16 / sizeof(T), of
// one u and many v.
template <typename T, bool PLANES>
struct RunOut {
    T *p;
    int64_t stride;
    uint32_t u, len;
    const Planes &pl;
    bool whole;
    __device__ __forceinline__ RunOut(T *base, const Planes &planes, uint32_t u_, uint32_t len_)
        : p(base + planes.run<PLANES>(u_)), stride(planes.stride<PLANES>()), u(u_), len(len_), pl(planes),
          whole(planes.whole<PLANES>(u_, len_))  // (eight points in a plane: more than fp32's four need)
    {
    }
    __device__ __forceinline__ void put(int64_t v, const u32x4 &w, bool nt = false) const
    {
        constexpr int n = 16 / (int)sizeof(T);
        T *q = p + v * stride;
        if (whole) {
            if (nt) store_as<true>(q, w);
            else store_as<false>(q, w);
            return;
        }
        const int64_t at0 = pl.run<PLANES>(u);
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (u + i < len) {
                T *to = q + (pl.run<PLANES>(u + i) - at0);
                if constexpr (sizeof(T) == 4) *(uint32_t *)to = w[i];
                else *(uint16_t *)to = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            }
    }
};

// One accumulator of the matrix cores to memory without LDS.  A lane holds column v = lane % 32 and four neighbouring rows
// u = 8 g + 4 (lane / 32) .. of it for g = 0 .. 3; lanes exchange halves, sixteens and eights until a store writes 64 or 128
// bytes of each v.
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// `f`: N neighbouring accumulators along u (1 or 2).  `p`: this lane's place, at frag_u<N>(lane) of their u and frag_v<N>(lane)
// of their v; `stride`: from v to v.  Two of them make whole lines of 128 bytes of 16-bit values.
template <typename T, int N>
__device__ __forceinline__ int frag_u(int lane)
{
    if constexpr (sizeof(T) == 4) return 8 * (lane >> 4 & 1) + 4 * (lane >> 5);
    else return 16 * (lane >> 4 & 1) + 8 * (lane >> 5) + (N == 2 ? 32 * (lane >> 3 & 1) : 0);
}

template <typename T, int N>
__device__ __forceinline__ int frag_v(int lane) { return sizeof(T) == 2 && N == 2 ? lane & 7 : lane & 15; }

// Lanes 8 .. 15 of each sixteen of `a` and 0 .. 7 of `b` change places.
__device__ __forceinline__ void swap8(uint32_t &a, uint32_t &b)
{
    const uint32_t x = (uint32_t)__builtin_amdgcn_update_dpp((int)a, (int)b, 0x128, 0xf, 0xc, false);
    b = (uint32_t)__builtin_amdgcn_update_dpp((int)b, (int)a, 0x128, 0xf, 0x3, false);
    a = x;
}

template <typename T, int N, bool NT>
__device__ __forceinline__ void store_frag(T *p, int64_t stride, const f32x4 (&f)[N][4])
{
    if constexpr (sizeof(T) == 2) {
        uint32_t w[N][4][2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float v[4] = {f[n][g][0], f[n][g][1], f[n][g][2], f[n][g][3]};
                Pack<T, 4> k;
                pack(v, k);
                w[n][g][0] = k.w[0];
                w[n][g][1] = k.w[1];
            }
            // halves: eight u of one g in each lane (g 0 and 2 below lane 32, 1 and 3 above); then the second sixteen
#pragma unroll
            for (int g = 0; g < 4; g += 2)
#pragma unroll
                for (int i = 0; i < 2; ++i) swap32(w[n][g][i], w[n][g + 1][i]);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) swap16(w[n][g][i], w[n][g + 2][i]);
        }
        if constexpr (N == 2)
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) swap8(w[0][g][i], w[1][g][i]);
#pragma unroll
        for (int g = 0; g < 4; g += 2)
#pragma unroll
            for (int n = 0; n < N; ++n)
                store_as<NT>(p + (8 * g + 8 * n) * stride, u32x4{w[n][g][0], w[n][g][1], w[n][g + 1][0], w[n][g + 1][1]});
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                uint32_t a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = __float_as_uint(f[n][g][i]);
                    b[i] = __float_as_uint(f[n][g + 1][i]);
                    swap16(a[i], b[i]);
                }
                store_as<NT>(p + 32 * n + 8 * g, u32x4{a[0], a[1], a[2], a[3]});
                store_as<NT>(p + 32 * n + 8 * g + 16 * stride, u32x4{b[0], b[1], b[2], b[3]});
            }
    }
}

// The same, element by element, for what lies below U and V.
template <typename T, bool PLANES>
__device__ __forceinline__ void store_frag_part(T *base, const Planes &pl, int lane, uint32_t u0, uint32_t U, uint32_t v0, uint32_t V, const f32x4 (&f)[4])
{
    const uint32_t v = v0 + (lane & 31);
    if (v >= V) return;
    T *row = base + (int64_t)v * pl.stride<PLANES>();
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t u = u0 + 8 * g + 4 * (lane >> 5) + e;
            if (u < U) store_elem(row, pl.run<PLANES>(u), f[g][e]);
        }
}

// One 32 x 32 x 16 product of the data type (operands travel as raw 16-bit patterns).
template <bool F16>
__device__ __forceinline__ f32x16 bwd_mma(bf16x8 a, bf16x8 b, f32x16 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const float f[2] = {a, b};
    if constexpr (F16) {
        Pack<f16_t, 2> p;
        pack(f, p);
        return p.w[0];
    } else {
        Pack<bf16_t, 2> p;
        pack(f, p);
        return p.w[0];
    }
}

// Four neighbouring values in the output's type.
template <typename T>
__device__ __forceinline__ void put4(unsigned char *to, const f32x4 &f)
{
    if constexpr (sizeof(T) == 4) {
        *(f32x4 *)to = f;
    } else {
        const float v[4] = {f[0], f[1], f[2], f[3]};
        Pack<T, 4> p;
        pack(v, p);
        *(u32x2 *)to = u32x2{p.w[0], p.w[1]};
    }
}

}  // namespace disco
