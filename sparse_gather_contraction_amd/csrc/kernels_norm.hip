// kernels_norm.hip — root-mean-square norm of x + residual, with an output in the data type or in 8 bits
// with scales, and the reader of the 8-bit form.
//
//   h = x + r;  rstd = (mean_d h^2 + eps)^(-1/2);  y = h rstd w
//   8 bits, per (n, group of channels, m):  scale = max(max |y| / qmax, 2^-126);  q = round(y / scale)
//
// Everything between the loads and the one rounding of each output is fp32: the sum h before it is
// rounded for storage, the mean of squares, y and the scales.  Memory traffic bounds every size beyond
// the smallest (4 to 7 flops an element), so each element is read once and held in registers from the
// sum to the write.  With a residual, 2x256x721x1440 bf16 takes 745-847 us from card to card (5.1-5.7 TB/s; a copy in
// the same 512-byte runs 790-870, a linear one 724-760), 4x32x181x360 fp32 19.4 us, rows of 512 bf16 176 us for
// 259200 (6.0 TB/s); 8 bits, 1x80x721x1440 bf16 117-121 us, 259200x512 fp16 without a residual 73 us (5.4 TB/s).
#include "kernels.hpp"
#include "norm.hpp"
#include "norm_device.hpp"

namespace disco {

namespace {

struct NormArgs {
    const void *x, *r, *w;
    void *y, *h;
    float *scale;
    int64_t N, M;
    int32_t D, wf32, group, ngroups, f8, lg, tiles_n;
    float eps, qmax;
};

// ---------------------------------------------------------------- columns (M > 1)

// A workgroup: 2^lg lanes along the points, `groups` threads along the channels, `CPT` channels a thread.
// LDS: [parts][P] partial sums (a part: a wave, or the threads of one g where those are more), [P] rstd, and for 8-bit outputs [ngroups][P] maxima.
template <typename T, int VEC, int CPT, bool RES, bool F8, bool NT>
__global__ __launch_bounds__(kNormMaxThreads) void norm_cols_kernel(NormArgs a)
{
    extern __shared__ float lds[];
    const int t = threadIdx.x, lane = t & ((1 << a.lg) - 1), g = t >> a.lg;
    const int P = VEC << a.lg, in_wave = a.lg < 6 ? 6 : a.lg, parts = blockDim.x >> in_wave, part = t >> in_wave;
    float *sums = lds, *rs = lds + parts * P;
    uint32_t *mx = (uint32_t *)(rs + P);
    const int64_t tile = NT ? blockIdx.x : xcd_tile(blockIdx.x, gridDim.x);
    const ColPos pos = col_pos(tile, lane, VEC, a.lg, a.tiles_n, a.N, a.M);
    const int c0 = g * CPT;
    const int64_t base = pos.n * a.D * a.M + pos.m;
    const T *x = (const T *)a.x + base, *r = (const T *)a.r + base;
    if constexpr (F8) {
        for (int i = t; i < a.ngroups * P; i += blockDim.x) mx[i] = 0;
    }

    float h[CPT][VEC];
    {
        Pack<T, VEC> px[CPT], pr[CPT];
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int64_t o = (int64_t)(c0 + j < a.D ? c0 + j : a.D - 1) * a.M;
            px[j] = load_pack<T, VEC>(x + o);
            if constexpr (RES) pr[j] = load_pack<T, VEC>(r + o);
        }
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            unpack(px[j], h[j]);
            if constexpr (RES) {
                float f[VEC];
                unpack(pr[j], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[j][e] += f[e];
            }
        }
    }
    float ss[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) ss[e] = 0.0f;
#pragma unroll
    for (int j = 0; j < CPT; ++j)
        if (c0 + j < a.D)
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss[e] = __builtin_fmaf(h[j][e], h[j][e], ss[e]);
    if (a.lg < 6)  // the wave's threads that hold the same points
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[e] = join_apart(ss[e], a.lg, AddOp());
    if (a.lg >= 6 || (t & 63) < (1 << a.lg))
#pragma unroll
        for (int e = 0; e < VEC; ++e) sums[part * P + lane * VEC + e] = ss[e];
    if constexpr (RES) {  // the stored sum leaves while the statistics are joined
        T *hs = (T *)a.h + base;
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (c0 + j < a.D) store_f32<T, VEC, NT>(hs + (int64_t)(c0 + j) * a.M, h[j]);
    }
    __syncthreads();
    for (int p = t; p < P; p += blockDim.x) {
        float s = 0.0f;
        for (int i = 0; i < parts; ++i) s += sums[i * P + p];
        rs[p] = rsqrtf(s / (float)a.D + a.eps);
    }
    __syncthreads();
    float rstd[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) rstd[e] = rs[lane * VEC + e];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
        const float w = load_weight<T>(a.w, a.wf32, c0 + j < a.D ? c0 + j : a.D - 1);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[j][e] = h[j][e] * rstd[e] * w;
    }
    if constexpr (!F8) {
        T *y = (T *)a.y + base;
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (c0 + j < a.D) store_f32<T, VEC, NT>(y + (int64_t)(c0 + j) * a.M, h[j]);
    } else {
        // a thread's channels share one scale: CPT divides 32, and 32 divides the group
        const int k = c0 < a.D ? c0 / a.group : 0;
        float m[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) m[e] = 0.0f;
#pragma unroll
        for (int j = 0; j < CPT; j += 2)  // an odd last channel is taken twice
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c0 + j < a.D) m[e] = max_abs(m[e], h[j][e], h[j + 1 < CPT && c0 + j + 1 < a.D ? j + 1 : j][e]);
        if (c0 < a.D)
#pragma unroll
            for (int e = 0; e < VEC; ++e) atomicMax(&mx[k * P + lane * VEC + e], abs_bits(m[e]));
        __syncthreads();
        if (c0 >= a.D) return;
        float s[VEC], inv[VEC], back[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const F8Scale f = f8_scale(__uint_as_float(mx[k * P + lane * VEC + e]), a.qmax);
            s[e] = f.scale;
            inv[e] = f.inv;
            back[e] = f.back;
        }
        if (c0 == k * a.group) store_f32<float, VEC>(a.scale + (pos.n * a.ngroups + k) * a.M + pos.m, s);
        uint8_t *q = (uint8_t *)a.y + base;
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (c0 + j < a.D) {
                float v[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = f8_quot(h[j][e], inv[e], back[e]);
                Pack<uint8_t, VEC> pq;
                pack_f8(v, a.f8, pq);
                store_pack<uint8_t, VEC, NT>(q + (int64_t)(c0 + j) * a.M, pq);
            }
    }
}

// ---------------------------------------------------------------- rows (M = 1)

// Joins a value over the 2^lg threads of a row: within a wave, then through LDS (one slot a wave).
template <typename Op>
__device__ __forceinline__ float row_join(float v, int lg, float *slots, Op op)
{
    v = join_run(v, lg, op);
    if (lg > 6) {  // uniform over the workgroup
        const int wave = threadIdx.x >> 6, per_row = 1 << (lg - 6), first = wave & ~(per_row - 1);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) slots[wave] = v;
        __syncthreads();
        v = slots[first];
        for (int i = 1; i < per_row; ++i) v = op(v, slots[first + i]);
    }
    return v;
}

// Zeroes what the thread holds beside another one, so that it adds nothing to a sum or a maximum.
template <int VEC>
__device__ __forceinline__ void drop_dup(float (&h)[VEC], int dup)
{
    if (dup)  // only the last vectors of a row
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = e < dup ? 0.0f : h[e];
}

// Stores the elements of a vector that no other thread holds.
template <typename T, int VEC, bool NT>
__device__ __forceinline__ void store_own(T *p, const Pack<T, VEC> &r, int dup)
{
    if (dup == 0) {
        store_pack<T, VEC, NT>(p, r);
    } else {
        const uint32_t per = 4 / sizeof(T);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (e >= dup) {
                if constexpr (sizeof(T) == 4) ((uint32_t *)p)[e] = r.w[e];
                else if constexpr (sizeof(T) == 2) ((uint16_t *)p)[e] = (uint16_t)(r.w[e / per] >> (16 * (e % per)));
                else ((uint8_t *)p)[e] = (uint8_t)(r.w[e / per] >> (8 * (e % per)));
            }
    }
}

// 2^lg threads a row, KPT vectors a thread.  Dynamic LDS: 8-bit outputs with groups that no run of lanes
// can join keep [rows][ngroups] maxima there.
template <typename T, int VEC, int KPT, bool RES, bool F8, bool NT>
__global__ __launch_bounds__(kNormMaxThreads) void norm_rows_kernel(NormArgs a)
{
    extern __shared__ uint32_t mx[];
    __shared__ float slots[kNormMaxThreads / 64];
    const int t = threadIdx.x, lanes = 1 << a.lg, tt = t & (lanes - 1), slot = t >> a.lg;
    const int64_t want = (int64_t)blockIdx.x * (blockDim.x >> a.lg) + slot;
    const int64_t row = want < a.N ? want : a.N - 1;  // a slot past the end repeats the last row
    const T *x = (const T *)a.x + row * a.D, *r = (const T *)a.r + row * a.D;
    RowPos pos[KPT];
    float h[KPT][VEC];
    {
        Pack<T, VEC> px[KPT], pr[KPT];
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            pos[k] = row_pos(k * lanes + tt, VEC, a.D);
            px[k] = load_pack<T, VEC>(x + pos[k].c);
            if constexpr (RES) pr[k] = load_pack<T, VEC>(r + pos[k].c);
        }
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            unpack(px[k], h[k]);
            if constexpr (RES) {
                float f[VEC];
                unpack(pr[k], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[k][e] += f[e];
            }
            drop_dup(h[k], pos[k].dup);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < KPT; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = __builtin_fmaf(h[k][e], h[k][e], ss);
    ss = row_join(ss, a.lg, slots, AddOp());
    const float rstd = rsqrtf(ss / (float)a.D + a.eps);
    if constexpr (RES) {
        T *hs = (T *)a.h + row * a.D;
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            Pack<T, VEC> p;
            pack(h[k], p);
            store_own<T, VEC, NT>(hs + pos[k].c, p, pos[k].dup);
        }
    }
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        float w[VEC];
        if (a.wf32) load_f32<float, VEC>((const float *)a.w + pos[k].c, w);
        else load_f32<T, VEC>((const T *)a.w + pos[k].c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[k][e] = h[k][e] * rstd * w[e];
    }
    if constexpr (!F8) {
        T *y = (T *)a.y + row * a.D;
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            Pack<T, VEC> p;
            pack(h[k], p);
            store_own<T, VEC, NT>(y + pos[k].c, p, pos[k].dup);
        }
    } else {
        float m[KPT];
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            drop_dup(h[k], pos[k].dup);  // a NaN rstd or weight has come back into the zeroes
            m[k] = 0.0f;
#pragma unroll
            for (int e = 0; e < VEC; e += 2) m[k] = max_abs(m[k], h[k][e], h[k][e + 1 < VEC ? e + 1 : e]);
        }
        const int gv = a.group / VEC;  // vectors of a group
        if (a.ngroups == 1) {
            float all = m[0];
#pragma unroll
            for (int k = 1; k < KPT; ++k) all = MaxOp()(all, m[k]);
            all = row_join(all, a.lg, slots, MaxOp());
#pragma unroll
            for (int k = 0; k < KPT; ++k) m[k] = all;
        } else if ((gv & (gv - 1)) == 0 && gv <= (lanes < 64 ? lanes : 64)) {
            const int lgv = 31 - __builtin_clz(gv);
#pragma unroll
            for (int k = 0; k < KPT; ++k) m[k] = join_run(m[k], lgv, MaxOp());
        } else {
            uint32_t *mine = mx + slot * a.ngroups;
            for (int i = t; i < (int)(blockDim.x >> a.lg) * a.ngroups; i += blockDim.x) mx[i] = 0;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < KPT; ++k)
                if (pos[k].dup < VEC) atomicMax(&mine[((k * lanes + tt) * VEC) / a.group], abs_bits(m[k]));
            __syncthreads();
#pragma unroll
            for (int k = 0; k < KPT; ++k)
                if (pos[k].dup < VEC) m[k] = __uint_as_float(mine[((k * lanes + tt) * VEC) / a.group]);
        }
        uint8_t *q = (uint8_t *)a.y + row * a.D;
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            if (pos[k].dup >= VEC) continue;
            const int c = (k * lanes + tt) * VEC, grp = a.ngroups == 1 ? 0 : c / a.group;
            const F8Scale f = f8_scale(m[k], a.qmax);
            if (c == grp * a.group) a.scale[row * a.ngroups + grp] = f.scale;
            float v[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = f8_quot(h[k][e], f.inv, f.back);
            Pack<uint8_t, VEC> pq;
            pack_f8(v, a.f8, pq);
            store_own<uint8_t, VEC, NT>(q + pos[k].c, pq, pos[k].dup);
        }
    }
}

// ---------------------------------------------------------------- more channels than registers hold

// 2^lg points at a time; the threads walk the channels once for the sum, once for the scales of an 8-bit
// output and once for the write, re-reading x and r through the caches.
template <typename T, bool RES, bool F8>
__global__ __launch_bounds__(kNormMaxThreads) void norm_loop_kernel(NormArgs a)
{
    extern __shared__ float lds[];  // [groups][P], [P], 8-bit: [ngroups][P] of the current channels' scales
    const int t = threadIdx.x, P = 1 << a.lg, lane = t & (P - 1), g = t >> a.lg, groups = blockDim.x >> a.lg;
    float *sums = lds, *rs = lds + groups * P;
    const ColPos pos = col_pos(blockIdx.x, lane, 1, a.lg, 0, a.N, a.M);
    const int64_t base = pos.n * a.D * a.M + pos.m;
    const T *x = (const T *)a.x + base, *r = (const T *)a.r + base;
    auto value = [&](int c) {
        float v = load_elem(x, (int64_t)c * a.M);
        if constexpr (RES) v += load_elem(r, (int64_t)c * a.M);
        return v;
    };
    float ss = 0.0f;
    for (int c = g; c < a.D; c += groups) {
        const float v = value(c);
        ss = __builtin_fmaf(v, v, ss);
    }
    sums[g * P + lane] = ss;
    __syncthreads();
    // a tree over the threads of a point: `groups` is a power of two
    for (int o = groups >> 1; o > 0; o >>= 1) {
        if (g < o) sums[g * P + lane] += sums[(g + o) * P + lane];
        __syncthreads();
    }
    if (g == 0) rs[lane] = rsqrtf(sums[lane] / (float)a.D + a.eps);
    __syncthreads();
    const float rstd = rs[lane];
    if constexpr (!F8) {
        for (int c = g; c < a.D; c += groups) {
            const float v = value(c);
            if constexpr (RES) store_elem((T *)a.h + base, (int64_t)c * a.M, v);
            store_elem((T *)a.y + base, (int64_t)c * a.M, v * rstd * load_weight<T>(a.w, a.wf32, c));
        }
    } else {
        float *mx = sums;  // [groups][P]: the group's maximum over the threads
        for (int k = 0; k < a.ngroups; ++k) {
            const int lo = k * a.group, hi = lo + a.group < a.D ? lo + a.group : a.D;
            float m = 0.0f;
            for (int c = lo + g; c < hi; c += groups) {
                const float y = value(c) * rstd * load_weight<T>(a.w, a.wf32, c);
                m = max_abs(m, y, y);
            }
            __syncthreads();
            mx[g * P + lane] = m;
            __syncthreads();
            for (int o = groups >> 1; o > 0; o >>= 1) {
                if (g < o) mx[g * P + lane] = MaxOp()(mx[g * P + lane], mx[(g + o) * P + lane]);
                __syncthreads();
            }
            const F8Scale f = f8_scale(mx[lane], a.qmax);
            if (g == 0) a.scale[(pos.n * a.ngroups + k) * a.M + pos.m] = f.scale;
            for (int c = lo + g; c < hi; c += groups) {
                const float v = value(c);
                if constexpr (RES) store_elem((T *)a.h + base, (int64_t)c * a.M, v);
                const float q1[1] = {f8_quot(v * rstd * load_weight<T>(a.w, a.wf32, c), f.inv, f.back)};
                Pack<uint8_t, 1> pq;
                pack_f8(q1, a.f8, pq);
                store_pack<uint8_t, 1>((uint8_t *)a.y + base + (int64_t)c * a.M, pq);
            }
        }
    }
}

template <typename T, bool RES, bool F8, bool NT>
void launch_nt(const NormArgs &a, const NormGeom &g, size_t lds, hipStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    const dim3 grid((uint32_t)g.tiles), block(g.threads);
#define ROWS(KPT) norm_rows_kernel<T, V, KPT, RES, F8, NT><<<grid, block, lds, s>>>(a)
#define COLS(CPT) norm_cols_kernel<T, V, CPT, RES, F8, NT><<<grid, block, lds, s>>>(a)
    if (g.rows) {
        if (g.per == 1) ROWS(1);
        else if (g.per == 2) ROWS(2);
        else ROWS(4);
    } else {
        if (g.per == 1) COLS(1);
        else if (g.per == 2) COLS(2);
        else if (g.per == 4) COLS(4);
        else COLS(8);
    }
#undef ROWS
#undef COLS
}

template <typename T, bool RES, bool F8>
hipError_t launch_t(const NormArgs &a, const NormGeom &g, hipStream_t s)
{
    const dim3 grid((uint32_t)g.tiles), block(g.threads);
    const size_t lds = norm_lds(g, F8 ? a.ngroups : 0);
    const int64_t out = a.N * a.D * a.M * ((RES ? sizeof(T) : 0) + (F8 ? 1 : sizeof(T)));
    const int64_t run = (g.rows ? a.D : a.M) * (int64_t)(RES || !F8 ? sizeof(T) : 1);
#define COLS(CPT) norm_cols_kernel<T, 1, CPT, RES, F8, false><<<grid, block, lds, s>>>(a)
    if (g.loop) {
        norm_loop_kernel<T, RES, F8><<<grid, block, lds, s>>>(a);
    } else if (g.vec > 1) {
        if (stream_stores(g.rows, out, run, a.y, a.h)) launch_nt<T, RES, F8, true>(a, g, lds, s);
        else launch_nt<T, RES, F8, false>(a, g, lds, s);
    } else if (g.rows) {
        norm_rows_kernel<T, 1, 1, RES, F8, false><<<grid, block, lds, s>>>(a);
    } else {
        if (g.per == 1) COLS(1);
        else if (g.per == 2) COLS(2);
        else if (g.per == 4) COLS(4);
        else COLS(8);
    }
#undef COLS
    return hipGetLastError();
}

template <typename T>
hipError_t launch_r(const NormArgs &a, const NormGeom &g, bool res, bool f8, hipStream_t s)
{
    if (res) return f8 ? launch_t<T, true, true>(a, g, s) : launch_t<T, true, false>(a, g, s);
    return f8 ? launch_t<T, false, true>(a, g, s) : launch_t<T, false, false>(a, g, s);
}

}  // namespace

hipError_t launch_norm(const NormLaunch &l, hipStream_t s)
{
    const NormGeom g = norm_geom(l.N, l.D, l.M, l.dtype == 0 ? 4 : 2, false);
    NormArgs a;
    a.x = l.x; a.r = l.r; a.w = l.w; a.y = l.y; a.h = l.h; a.scale = l.scale;
    a.N = l.N; a.M = l.M; a.D = (int32_t)l.D; a.wf32 = l.wf32;
    a.group = l.group; a.ngroups = l.ngroups; a.f8 = l.f8; a.lg = g.lg; a.tiles_n = g.tiles_n;
    a.eps = l.eps; a.qmax = l.f8 == 1 ? 57344.0f : 448.0f;
    const bool res = l.r != nullptr, f8 = l.f8 >= 0;
    return l.dtype == 0 ? launch_r<float>(a, g, res, f8, s)
         : l.dtype == 1 ? launch_r<bf16_t>(a, g, res, f8, s)
                        : launch_r<f16_t>(a, g, res, f8, s);
}

// ---------------------------------------------------------------- reader of the 8-bit form

namespace {

struct DequantArgs {
    const uint8_t *q;
    const float *scale;
    void *out;
    int64_t N, M;
    int32_t D, group, ngroups, f8, lg, tiles_n, chunks;
};

// columns: a thread holds VEC points of CPT channels under one scale, which it loads once; nothing is joined, so a
// workgroup is four waves of as many channel blocks.  1x80x721x1440 to bf16 38.5 us (6.6 TB/s).
template <typename T, int VEC, int CPT, bool NT>
__global__ __launch_bounds__(256) void dequant_cols_kernel(DequantArgs a)
{
    const int lane = threadIdx.x & ((1 << a.lg) - 1), g = threadIdx.x >> a.lg;
    const uint32_t id = (uint32_t)xcd_tile(blockIdx.x, gridDim.x);  // 1x80x721x1440 bf16: 38.5 against 42.0 us
    const int64_t tile = id / (uint32_t)a.chunks;
    const int chunk = id % (uint32_t)a.chunks;
    const int c0 = (chunk * (int)(blockDim.x >> a.lg) + g) * CPT;
    if (c0 >= a.D) return;
    const ColPos pos = col_pos(tile, lane, VEC, a.lg, a.tiles_n, a.N, a.M);
    const int k = c0 / a.group;
    const int64_t base = pos.n * a.D * a.M + pos.m;
    Pack<uint8_t, VEC> pq[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j)
        pq[j] = load_pack<uint8_t, VEC>(a.q + base + (int64_t)(c0 + j < a.D ? c0 + j : a.D - 1) * a.M);
    float s[VEC];
    load_f32<float, VEC>(a.scale + (pos.n * a.ngroups + k) * a.M + pos.m, s);
    T *out = (T *)a.out + base;
#pragma unroll
    for (int j = 0; j < CPT; ++j)
        if (c0 + j < a.D) {
            float v[VEC];
            unpack_f8(pq[j], a.f8, v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] *= s[e];
            store_f32<T, VEC, NT>(out + (int64_t)(c0 + j) * a.M, v);
        }
}

// rows: 2^lg threads a row, each walking its vectors.  259200x512 to fp16 60 us (6.7 TB/s) where the input is in the
// last-level cache, 70 where it is not.
template <typename T, int VEC, bool NT>
__global__ __launch_bounds__(256) void dequant_rows_kernel(DequantArgs a)
{
    const int lanes = 1 << a.lg, tt = threadIdx.x & (lanes - 1), slot = threadIdx.x >> a.lg;
    const int64_t row = (int64_t)blockIdx.x * (256 >> a.lg) + slot;
    if (row >= a.N) return;
    const int nv = (a.D + VEC - 1) / VEC;
    for (int v = tt; v < nv; v += lanes) {
        const RowPos pos = row_pos(v, VEC, a.D);
        const Pack<uint8_t, VEC> pq = load_pack<uint8_t, VEC>(a.q + row * a.D + pos.c);
        const float s = a.scale[row * a.ngroups + (v * VEC) / a.group];
        float f[VEC];
        unpack_f8(pq, a.f8, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] *= s;
        T *out = (T *)a.out + row * a.D + pos.c;
        Pack<T, VEC> p;
        pack(f, p);
        store_own<T, VEC, NT>(out, p, pos.dup);  // what is held twice may belong to another group's scale
    }
}

template <typename T>
hipError_t launch_dequant_t(DequantArgs a, const DequantGeom &g, hipStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    const dim3 grid((uint32_t)g.blocks);
    // A wave's runs are 1 KiB here, so sectors that two tiles share are few: stores past the L2 gain with them too
    // (1x512x361x720 72 against 90 us, rows of 512 61 against 72 us).
    const bool nt = a.N * a.D * a.M * (int64_t)sizeof(T) > kStreamRows;
    if (a.M == 1) {
        if (!g.vec) dequant_rows_kernel<T, 1, false><<<grid, 256, 0, s>>>(a);
        else if (nt) dequant_rows_kernel<T, V, true><<<grid, 256, 0, s>>>(a);
        else dequant_rows_kernel<T, V, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (!g.vec) dequant_cols_kernel<T, 1, kDequantCpt, false><<<grid, 256, 0, s>>>(a);
        else if (nt) dequant_cols_kernel<T, V, kDequantCpt, true><<<grid, 256, 0, s>>>(a);
        else dequant_cols_kernel<T, V, kDequantCpt, false><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dequant(const DequantLaunch &l, hipStream_t s)
{
    DequantArgs a;
    a.q = l.q; a.scale = l.scale; a.out = l.out;
    a.N = l.N; a.M = l.M; a.D = (int32_t)l.D; a.group = l.group; a.ngroups = l.ngroups; a.f8 = l.f8;
    const DequantGeom g = dequant_geom(l.N, l.D, l.M, l.dtype == 0 ? 4 : 2);
    a.lg = g.lg; a.tiles_n = g.tiles_n; a.chunks = g.chunks;
    return l.dtype == 0 ? launch_dequant_t<float>(a, g, s)
         : l.dtype == 1 ? launch_dequant_t<bf16_t>(a, g, s)
                        : launch_dequant_t<f16_t>(a, g, s);
}

}  // namespace disco
