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

constexpr uint32_t kLinOob = 0x80000000u;  // beyond every buffer used here: the load gives zeros

// Points of a tensor whose point axis is contiguous within planes of M, J channels a plane: element (j, g).
struct Planes {
    FastDiv by_m;
    int64_t M, J;
    __device__ __forceinline__ int64_t at(int64_t j, uint32_t g) const
    {
        const uint32_t n = by_m.div(g);
        return ((int64_t)n * J + j) * M + (g - n * (uint32_t)M);
    }
    // whether points g .. g + 7 lie in one plane
    __device__ __forceinline__ bool whole(uint32_t g) const
    {
        return g - by_m.div(g) * (uint32_t)M + 8 <= (uint32_t)M;
    }
};

// Eight 16-bit elements (j, c .. c + 7) of a tensor whose axis c lies together, `len` long: PLANES: c are points in
// planes, else (j, c) lies at j ld + c.  Zeros where c passes len.  Rows j are the caller's to bound.
template <bool PLANES>
__device__ __forceinline__ u32x4 load_run(const uint16_t *base, const Planes &pl, int64_t ld, int64_t j, uint32_t c, uint32_t len)
{
    if (c + 8 <= len && (!PLANES || pl.whole(c))) return load_as<false, u32x4>(base + (PLANES ? pl.at(j, c) : j * ld + c));
    u32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < len) r[i / 2] |= (uint32_t)base[PLANES ? pl.at(j, c + i) : j * ld + c + i] << (16 * (i & 1));
    return r;
}

// Elements (v, u .. u + n-1), n = 16 / sizeof(T), of an output whose axis u lies together.
template <typename T, bool PLANES>
__device__ __forceinline__ void store_run(T *base, const Planes &pl, int64_t ld, int64_t v, uint32_t u, uint32_t len, const u32x4 &w)
{
    constexpr int n = 16 / (int)sizeof(T);
    if (u + n <= len && (!PLANES || pl.whole(u))) {  // (eight points in a plane: more than fp32's four need)
        store_as<false>(base + (PLANES ? pl.at(v, u) : v * ld + u), w);
        return;
    }
#pragma unroll
    for (int i = 0; i < n; ++i)
        if (u + i < len) {
            T *p = base + (PLANES ? pl.at(v, u + i) : v * ld + u + i);
            if constexpr (sizeof(T) == 4) *(uint32_t *)p = w[i];
            else *(uint16_t *)p = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
}

}  // namespace disco
