// kernels_norm_bwd.hip — backward of the root-mean-square norm.
//
// With h the stored sum, g = gy w, rstd = (mean_d h^2 + eps)^(-1/2):
//   gx = rstd (g - u c) (+ gh, the gradient that reaches h past the norm),  u = h rstd,  c = rstd mean_d(g h)
//   dw[d] = sum over all points of gy u
// u is of the order of 1 and c of the order of g, so nothing on the way leaves fp32's range where h^2 does not
// (rstd^3 does: from |h| = 2^42 on it has no normal fp32 value).
//
// Each element of h, gy and gh is read once: both sums over the channels are taken while the tile lies in
// registers.  A workgroup keeps its threads' share of the channels for its whole life, so dw is summed in
// registers over the workgroup's tiles (the terms and their sum in fp64), then over its lanes, and
// the workgroups' partial rows are summed in fp64 by a second launch.  Rows too long for that have dw summed by a
// launch of its own (dw_rows_kernel).  Every order is fixed, so results are bitwise reproducible.
//
// Memory bounds it: 2x256x721x1440 bf16 with gh 781-862 us from card to card (4.9-5.4 TB/s; a copy in the same
// 256-byte runs takes 815-930), 259200x512 bf16 195 us (5.4 TB/s), 4x32x181x360 fp32 21.5 us and 3.8 of the second launch.
#include "kernels.hpp"
#include "norm.hpp"
#include "norm_device.hpp"

namespace disco {

namespace {

struct BwdArgs {
    const void *h, *gy, *gh, *w;
    void *gx;
    part_t *partial;
    float *rstd;   // long rows: rstd of each row, for the launch that sums dw
    void *dw;      // not null: the sums of the launch's one workgroup, or one chunk of rows, are dw itself
    int64_t N, M, tiles;
    int32_t D, wf32, lg, tiles_n;
    float eps;
};

// v, which the compiler takes for a new value: addresses made from it are made where they are used, and hold no
// registers from one tile to the next.
__device__ __forceinline__ int fresh(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// The sum for channel c of workgroup or chunk `part`: its entry of the partial sums, or dw.
template <typename T>
__device__ __forceinline__ void store_dw(const BwdArgs &a, int part, int c, double s)
{
    if (!a.dw) a.partial[(int64_t)part * a.D + c] = s;
    else if (a.wf32) ((float *)a.dw)[c] = (float)s;
    else store_elem((T *)a.dw, c, (float)s);
}

// Columns (M > 1): the forward's tiles.  LDS: [parts][P] sums of h^2, [parts][P] of g h, [P] rstd,
// [P] c; at the end [waves of one g][channels] fp64 of dw.
template <typename T, int VEC, int CPT, bool RES, bool NT>
__global__ __launch_bounds__(kNormMaxThreads) void bwd_cols_kernel(BwdArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int t = threadIdx.x, lane = t & ((1 << a.lg) - 1), g = t >> a.lg;
    const int P = VEC << a.lg, groups = blockDim.x >> a.lg;
    const int lg6 = a.lg < 6 ? 6 : a.lg, parts = blockDim.x >> lg6, part = t >> lg6;
    float *s_hh = lds, *s_gh = lds + parts * P, *rs = lds + 2 * parts * P, *cs = rs + P;
    const int c0 = g * CPT;
    float w[CPT];
    double acc[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
        w[j] = c0 + j < a.D ? load_weight<T>(a.w, a.wf32, c0 + j) : 0.0f;
        acc[j] = 0.0;
    }
    Pack<T, VEC> ph[CPT], pg[CPT], pr[CPT];
    ColPos pos = {0, 0, 0};
    int64_t base = 0;
    auto load_tile = [&](int64_t i) {
        pos = col_pos(NT ? i : xcd_tile(i, a.tiles), lane, VEC, a.lg, a.tiles_n, a.N, a.M);
        base = pos.n * a.D * a.M + pos.m;
        const int c = fresh(c0);
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int64_t o = base + (int64_t)(c + j < a.D ? c + j : a.D - 1) * a.M;
            ph[j] = load_pack<T, VEC>((const T *)a.h + o);
            pg[j] = load_pack<T, VEC>((const T *)a.gy + o);
        }
    };
    if (blockIdx.x < a.tiles) load_tile(blockIdx.x);
    for (int64_t i = blockIdx.x; i < a.tiles; i += gridDim.x) {
        float hh[VEC], gh[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) hh[e] = gh[e] = 0.0f;
        if (c0 + CPT > a.D)  // what was loaded in the place of channels past the end adds nothing
#pragma unroll
            for (int j = 0; j < CPT; ++j)
                if (c0 + j >= a.D) ph[j] = pg[j] = {};
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            float h[VEC], gy[VEC];
            unpack(ph[j], h);
            unpack(pg[j], gy);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                hh[e] = __builtin_fmaf(h[e], h[e], hh[e]);
                gh[e] = __builtin_fmaf(gy[e] * w[j], h[e], gh[e]);
            }
        }
        if (a.lg < 6)  // the wave's threads that hold the same points
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                hh[e] = join_apart(hh[e], a.lg, AddOp());
                gh[e] = join_apart(gh[e], a.lg, AddOp());
            }
        if (a.lg >= 6 || (t & 63) < (1 << a.lg))
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s_hh[part * P + lane * VEC + e] = hh[e];
                s_gh[part * P + lane * VEC + e] = gh[e];
            }
        __syncthreads();
        for (int p = t; p < P; p += blockDim.x) {
            float u = 0.0f, v = 0.0f;
            for (int i = 0; i < parts; ++i) {
                u += s_hh[i * P + p];
                v += s_gh[i * P + p];
            }
            const float r = rsqrtf(u / (float)a.D + a.eps);
            rs[p] = r;
            cs[p] = r * (v / (float)a.D);
        }
        __syncthreads();
        // gh is asked for only now: loaded with the others it takes registers from them and bandwidth at the
        // moment when the sums wait for h and gy (883 against 864 us at 2x256x721x1440 bf16, next tile not yet
        // asked for early).
        if constexpr (RES) {
            const int c = fresh(c0);
#pragma unroll
            for (int j = 0; j < CPT; ++j)
                pr[j] = load_pack<T, VEC>((const T *)a.gh + base + (int64_t)(c + j < a.D ? c + j : a.D - 1) * a.M);
        }
        float rstd[VEC], c[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            rstd[e] = rs[lane * VEC + e];
            c[e] = cs[lane * VEC + e];
        }
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            keep_packed(ph[j]);
            keep_packed(pg[j]);
        }
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            float h[VEC], gy[VEC], o[VEC];
            unpack(ph[j], h);
            unpack(pg[j], gy);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float u = h[e] * rstd[e];
                acc[j] = e >= pos.dup ? __builtin_fma((double)gy[e], (double)u, acc[j]) : acc[j];
                o[e] = rstd[e] * (gy[e] * w[j] - u * c[e]);
            }
            if constexpr (RES) {
                float r[VEC];
                unpack(pr[j], r);
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] += r[e];
            }
            pack(o, pr[j]);
            keep_here(pr[j]);  // one channel's fp32 values at a time
            keep_here(acc[j]);
        }
        // The next tile is asked for before this one's stores, in the registers that this one has left.
        T *gx = (T *)a.gx + base;
        if (i + gridDim.x < a.tiles) load_tile(i + gridDim.x);
        const int c1 = fresh(c0);
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (c1 + j < a.D) store_pack<T, VEC, NT>(gx + (int64_t)(c1 + j) * a.M, pr[j]);
    }
    const int in_wave = a.lg < 6 ? a.lg : 6, waves = a.lg > 6 ? 1 << (a.lg - 6) : 1, width = groups * CPT;
#pragma unroll
    for (int j = 0; j < CPT; ++j) acc[j] = join_run(acc[j], in_wave, AddOp());
    double *sum = (double *)lds;
    __syncthreads();
    if ((lane & ((1 << in_wave) - 1)) == 0)
#pragma unroll
        for (int j = 0; j < CPT; ++j) sum[(lane >> 6) * width + c0 + j] = acc[j];
    __syncthreads();
    for (int c = t; c < a.D; c += blockDim.x) {
        double s = sum[c];
        for (int i = 1; i < waves; ++i) s += sum[i * width + c];
        store_dw<T>(a, blockIdx.x, c, s);
    }
}

struct Sum2 {
    float u, v;
};

// Two sums over the 2^lg threads of a row.
__device__ __forceinline__ Sum2 row_sum2(Sum2 s, int lg, Sum2 *slots)
{
    s.u = join_run(s.u, lg, AddOp());
    s.v = join_run(s.v, lg, AddOp());
    if (lg > 6) {  // uniform over the workgroup
        const int wave = threadIdx.x >> 6, per_row = 1 << (lg - 6), first = wave & ~(per_row - 1);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) slots[wave] = s;
        __syncthreads();
        s = slots[first];
        for (int i = 1; i < per_row; ++i) {
            s.u += slots[first + i].u;
            s.v += slots[first + i].v;
        }
    }
    return s;
}

// Rows (M = 1).  dw is summed here, but for four vectors of 16 bits a thread: they do not have the registers for fp64
// sums and keep each row's rstd for dw_rows_kernel.
// Dynamic LDS: [rows][D] fp64 for the join of dw where a workgroup holds several rows; four vectors of fp32 a thread keep
// the weights of the first three there, each thread its own, in the place of registers that the sums of dw take
// (20000x10000 fp32 597 against 707 us, 16000x16384 778 against 840).
template <typename T, int VEC, int KPT, bool RES, bool NT>
__global__ __launch_bounds__(kNormMaxThreads) void bwd_rows_kernel(BwdArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    __shared__ Sum2 slots[kNormMaxThreads / 64];
    const int t = threadIdx.x, lanes = 1 << a.lg, tt = t & (lanes - 1), slot = t >> a.lg;
    const int rows = blockDim.x >> a.lg;
    RowPos pos[KPT];
    constexpr bool DW = KPT * VEC <= 16;
    constexpr int LW = KPT == 4 && VEC == 4 ? kBwdLdsWeights : 0;
    float w[KPT - LW][VEC];
    f32x4 *const lw = (f32x4 *)lds + t;
    auto weight = [&](int k, float (&f)[VEC]) {
        if constexpr (LW > 0)
            if (k < LW) {
                const f32x4 v = lw[k * blockDim.x];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = v[e];
                return;
            }
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = w[k - LW][e];
    };
    double acc[KPT][VEC];
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        pos[k] = row_pos(k * lanes + tt, VEC, a.D);
        float f[VEC];
        if (a.wf32) load_f32<float, VEC>((const float *)a.w + pos[k].c, f);
        else load_f32<T, VEC>((const T *)a.w + pos[k].c, f);
        if constexpr (LW > 0)
            if (k < LW) lw[k * blockDim.x] = f32x4{f[0], f[1], f[2], f[3]};
        if (k >= LW)
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[k - LW][e] = f[e];
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[k][e] = 0;
    }
    Pack<T, VEC> ph[KPT], pg[KPT], pr[KPT];
    bool live = false;
    int64_t row = 0, base = 0;
    auto load_tile = [&](int64_t tile) {
        const int64_t want = tile * rows + slot;
        live = want < a.N;
        row = live ? want : a.N - 1;  // a slot past the end repeats the last row
        base = row * a.D;
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            ph[k] = load_pack<T, VEC>((const T *)a.h + base + pos[k].c);
            pg[k] = load_pack<T, VEC>((const T *)a.gy + base + pos[k].c);
        }
    };
    if (blockIdx.x < a.tiles) load_tile(blockIdx.x);
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        if constexpr (RES) {
#pragma unroll
            for (int k = 0; k < KPT; ++k) pr[k] = load_pack<T, VEC>((const T *)a.gh + base + pos[k].c);
        }
        Sum2 s = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            float h[VEC], gy[VEC], wk[VEC];
            unpack(ph[k], h);
            unpack(pg[k], gy);
            weight(k, wk);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e >= pos[k].dup) {
                    s.u = __builtin_fmaf(h[e], h[e], s.u);
                    s.v = __builtin_fmaf(gy[e] * wk[e], h[e], s.v);
                }
        }
        s = row_sum2(s, a.lg, slots);
        const float rstd = rsqrtf(s.u / (float)a.D + a.eps), c = rstd * (s.v / (float)a.D);
        if constexpr (!DW)
            if (tt == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            keep_packed(ph[k]);
            keep_packed(pg[k]);
        }
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            float h[VEC], gy[VEC], wk[VEC], o[VEC];
            unpack(ph[k], h);
            unpack(pg[k], gy);
            weight(k, wk);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float u = h[e] * rstd;
                if constexpr (DW) acc[k][e] = live && e >= pos[k].dup ? __builtin_fma((double)gy[e], (double)u, acc[k][e]) : acc[k][e];
                o[e] = rstd * (gy[e] * wk[e] - u * c);
            }
            if constexpr (RES) {
                float r[VEC];
                unpack(pr[k], r);
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] += r[e];
            }
            pack(o, pr[k]);
            keep_here(pr[k]);
            if constexpr (DW)
#pragma unroll
                for (int e = 0; e < VEC; ++e) keep_here(acc[k][e]);
        }
        T *gx = (T *)a.gx + base;
        if (tile + gridDim.x < a.tiles) load_tile(tile + gridDim.x);  // before this row's stores, as in columns
#pragma unroll
        for (int k = 0; k < KPT; ++k)
            if (pos[k].dup < VEC) store_pack<T, VEC, NT>(gx + pos[k].c, pr[k]);
    }
    if constexpr (!DW) return;
    if (rows > 1) {
        double *sum = (double *)lds;
#pragma unroll
        for (int k = 0; k < KPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e >= pos[k].dup) sum[slot * a.D + pos[k].c + e] = acc[k][e];
        __syncthreads();
        for (int c = t; c < a.D; c += blockDim.x) {
            double s = 0.0;
            for (int i = 0; i < rows; ++i) s += sum[i * a.D + c];
            store_dw<T>(a, blockIdx.x, c, s);
        }
    } else {
#pragma unroll
        for (int k = 0; k < KPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e >= pos[k].dup) store_dw<T>(a, blockIdx.x, pos[k].c + e, acc[k][e]);
    }
}

// dw of long rows, in a launch of its own: a thread holds the fp64 sums of one vector of columns over a chunk of
// rows and reads h and gy once more.  Memory bounds it.  fp64 sums beside gx take more registers than there are (with
// fp32 ones, 20000x20000 bf16 took 1246 us with 216 bytes a thread spilled, both launches here 884), and a row of sums
// for each workgroup in device memory costs a read and a write of 8 bytes an element (2000x40000 bf16 620 us, here 455;
// the looping kernel with fp32 sums there 537).
template <typename T>
__global__ __launch_bounds__(kDwThreads) void dw_rows_kernel(BwdArgs a, int64_t rows)
{
    constexpr int VEC = 16 / (int)sizeof(T), U = 4;
    const int v = blockIdx.x * kDwThreads + threadIdx.x;
    if ((int64_t)v * VEC >= a.D) return;
    const RowPos pos = row_pos(v, VEC, a.D);
    const int64_t lo = blockIdx.y * rows, hi = lo + rows < a.N ? lo + rows : a.N;
    const T *hp = (const T *)a.h + pos.c, *gp = (const T *)a.gy + pos.c;
    double acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.0;
    for (int64_t i = lo; i < hi; i += U) {
        Pack<T, VEC> ph[U], pg[U];
        float rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = i + u < hi ? i + u : hi - 1;
            ph[u] = load_pack<T, VEC>(hp + row * a.D);
            pg[u] = load_pack<T, VEC>(gp + row * a.D);
            rstd[u] = a.rstd[row];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < hi) {
                float h[VEC], gy[VEC];
                unpack(ph[u], h);
                unpack(pg[u], gy);
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[e] = __builtin_fma((double)gy[e], (double)(h[e] * rstd[u]), acc[e]);
            }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        if (e >= pos.dup) store_dw<T>(a, blockIdx.y, pos.c + e, acc[e]);
}

// More channels than registers hold: the threads walk the channels twice.  Rows leave dw to dw_rows_kernel; else a
// workgroup's row of partial sums is kept in device memory, each entry by one thread.
template <typename T, bool RES>
__global__ __launch_bounds__(kNormMaxThreads) void bwd_loop_kernel(BwdArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int t = threadIdx.x, P = 1 << a.lg, lane = t & (P - 1), g = t >> a.lg, groups = blockDim.x >> a.lg;
    float *s_hh = lds, *s_gh = lds + groups * P;
    part_t *mine = a.partial + (int64_t)blockIdx.x * a.D;
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const ColPos pos = col_pos(tile, lane, 1, a.lg, 0, a.N, a.M);
        const int64_t base = pos.n * a.D * a.M + pos.m;
        const T *hp = (const T *)a.h + base, *gp = (const T *)a.gy + base;
        float hh = 0.0f, gh = 0.0f;
        for (int c = g; c < a.D; c += groups) {
            const float h = load_elem(hp, (int64_t)c * a.M), gy = load_elem(gp, (int64_t)c * a.M);
            hh = __builtin_fmaf(h, h, hh);
            gh = __builtin_fmaf(gy * load_weight<T>(a.w, a.wf32, c), h, gh);
        }
        __syncthreads();
        s_hh[g * P + lane] = hh;
        s_gh[g * P + lane] = gh;
        __syncthreads();
        for (int o = groups >> 1; o > 0; o >>= 1) {  // `groups` is a power of two
            if (g < o) {
                s_hh[g * P + lane] += s_hh[(g + o) * P + lane];
                s_gh[g * P + lane] += s_gh[(g + o) * P + lane];
            }
            __syncthreads();
        }
        const float rstd = rsqrtf(s_hh[lane] / (float)a.D + a.eps);
        const float k = rstd * (s_gh[lane] / (float)a.D);
        if (a.rstd && t == 0) a.rstd[tile] = rstd;
        for (int c = g; c < a.D; c += groups) {
            const float h = load_elem(hp, (int64_t)c * a.M), gy = load_elem(gp, (int64_t)c * a.M);
            const float u = h * rstd;
            float o = rstd * (gy * load_weight<T>(a.w, a.wf32, c) - u * k);
            if constexpr (RES) o += load_elem((const T *)a.gh + base, (int64_t)c * a.M);
            store_elem((T *)a.gx + base, (int64_t)c * a.M, o);
            if (a.rstd) continue;  // uniform
            // P <= 64 lanes of one wave walk together
            const double d = join_run(pos.dup ? 0.0 : (double)gy * (double)u, a.lg, AddOp());
            if (lane == 0) mine[c] = tile == blockIdx.x ? d : mine[c] + d;
        }
    }
}

// dw[c] = the sum of partial[0..parts)[c]: 16 columns a workgroup at a time, 64 threads a column, fp64.
template <typename O>
__global__ __launch_bounds__(kDwSumThreads) void dw_sum_kernel(const part_t *partial, int parts, int D, O *dw)
{
    __shared__ double part[16][kDwSumCols];
    const int col = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    for (int64_t c0 = (int64_t)blockIdx.x * kDwSumCols; c0 < D; c0 += (int64_t)gridDim.x * kDwSumCols) {
        const int64_t c = c0 + col;
        double s = 0.0;
        if (c < D) {
            for (int i = r0; i < parts; i += 8 * 64) {
                double v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = i + u * 64 < parts ? partial[(int64_t)(i + u * 64) * D + c] : 0.0;
#pragma unroll
                for (int u = 0; u < 8; ++u) s += v[u];
            }
        }
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if ((threadIdx.x & 63) < 16) part[threadIdx.x >> 6][col] = s;
        __syncthreads();
        if (r0 == 0 && c < D) {
            s = part[0][col];
#pragma unroll
            for (int i = 1; i < 16; ++i) s += part[i][col];
            store_elem(dw, c, (float)s);
        }
        __syncthreads();
    }
}

template <typename T, bool RES, bool NT>
void launch_nt(const BwdArgs &a, const NormGeom &g, int blocks, size_t lds, hipStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    const dim3 grid(blocks), block(g.threads);
#define ROWS(KPT) bwd_rows_kernel<T, V, KPT, RES, NT><<<grid, block, lds, s>>>(a)
#define COLS(CPT) bwd_cols_kernel<T, V, CPT, RES, NT><<<grid, block, lds, s>>>(a)
    if (g.rows) {
        if (g.per == 1) ROWS(1);
        else if (g.per == 2) ROWS(2);
        else ROWS(4);
    } else {
        if (g.per == 1) COLS(1);
        else if (g.per == 2) COLS(2);
        else COLS(4);
    }
#undef ROWS
#undef COLS
}

template <typename T, bool RES>
hipError_t launch_t(const BwdArgs &a, const NormGeom &g, int blocks, hipStream_t s)
{
    const dim3 grid(blocks), block(g.threads);
    const size_t lds = norm_bwd_lds(g, a.D);
    const bool nt = stream_stores(g.rows, a.N * a.D * a.M * (int64_t)sizeof(T), (g.rows ? a.D : a.M) * (int64_t)sizeof(T), a.gx, nullptr);
#define COLS(CPT) bwd_cols_kernel<T, 1, CPT, RES, false><<<grid, block, lds, s>>>(a)
    if (g.loop) {
        bwd_loop_kernel<T, RES><<<grid, block, lds, s>>>(a);
    } else if (g.vec > 1) {
        if (nt) launch_nt<T, RES, true>(a, g, blocks, lds, s);
        else launch_nt<T, RES, false>(a, g, blocks, lds, s);
    } else if (g.rows) {
        bwd_rows_kernel<T, 1, 1, RES, false><<<grid, block, lds, s>>>(a);
    } else {
        if (g.per == 1) COLS(1);
        else if (g.per == 2) COLS(2);
        else COLS(4);
    }
#undef COLS
    return hipGetLastError();
}

template <typename T>
hipError_t launch_r(BwdArgs a, const BwdPlan &p, bool res, void *dw, hipStream_t s)
{
    const hipError_t e = res ? launch_t<T, true>(a, p.g, p.blocks, s) : launch_t<T, false>(a, p.g, p.blocks, s);
    if (e != hipSuccess || !p.apart) return e;
    a.dw = p.parts == 1 ? dw : nullptr;
    dw_rows_kernel<T><<<dim3((uint32_t)p.dw_tiles, (uint32_t)p.parts), kDwThreads, 0, s>>>(a, p.dw_rows);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_bwd(const NormLaunch &l, hipStream_t s)
{
    const BwdPlan p = norm_bwd_plan(l.N, l.D, l.M, l.dtype == 0 ? 4 : 2);
    part_t *partial = (part_t *)l.workspace;
    if (p.blocks > 0) {
        BwdArgs a;
        a.dw = !p.apart && p.direct() ? l.dw : nullptr;
        a.h = l.x; a.gy = l.gy; a.gh = l.r; a.w = l.w; a.gx = l.y; a.partial = partial;
        a.rstd = p.apart ? (float *)(partial + (int64_t)p.parts * l.D) : nullptr;
        a.N = l.N; a.M = l.M; a.tiles = p.g.tiles;
        a.D = (int32_t)l.D; a.wf32 = l.wf32; a.lg = p.g.lg; a.tiles_n = p.g.tiles_n; a.eps = l.eps;
        const bool res = l.r != nullptr;
        const hipError_t e = l.dtype == 0 ? launch_r<float>(a, p, res, l.dw, s)
                           : l.dtype == 1 ? launch_r<bf16_t>(a, p, res, l.dw, s)
                                          : launch_r<f16_t>(a, p, res, l.dw, s);
        if (e != hipSuccess || p.direct()) return e;
    }
    const dim3 grid((uint32_t)dw_sum_blocks(l.D));
    if (l.wf32) dw_sum_kernel<float><<<grid, kDwSumThreads, 0, s>>>(partial, p.parts, (int)l.D, (float *)l.dw);
    else if (l.dtype == 1) dw_sum_kernel<bf16_t><<<grid, kDwSumThreads, 0, s>>>(partial, p.parts, (int)l.D, (bf16_t *)l.dw);
    else dw_sum_kernel<f16_t><<<grid, kDwSumThreads, 0, s>>>(partial, p.parts, (int)l.D, (f16_t *)l.dw);
    return hipGetLastError();
}

}  // namespace disco
