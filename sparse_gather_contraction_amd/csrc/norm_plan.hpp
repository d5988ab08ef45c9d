// norm_plan.hpp — launch geometry and index arithmetic of the norm kernels (host and device).
//
// A tensor is seen as (N, D, M): N the product of the sizes before the normalised axis, D that axis, M
// the product of the sizes after it; element (n, d, m) lies at (n D + d) M + m.  Two layouts of work:
//   columns (M > 1): a workgroup holds a tile of P consecutive points (n, m) with all their D channels;
//     thread (g, lane) holds channels g*per .. g*per+per-1 of the points lane*vec .. lane*vec+vec-1.
//   rows (M = 1): `lanes` threads hold one row, thread t the vectors t, t + lanes, ... of `vec` elements.
// A vector that would pass the end of its run is moved back to end there; `dup` says how many of its
// leading elements are held twice.  So every access is a whole vector inside the tensor, at any size.
#pragma once

#include <cstddef>
#include <cstdint>

#if defined(__HIPCC__)
#define DISCO_HD __host__ __device__ __forceinline__
#else
#define DISCO_HD inline
#endif

namespace disco {

struct NormGeom {
    int32_t rows = 0;      // 1: rows layout
    int32_t loop = 0;      // 1: the channels pass the threads' registers; the looping kernels
    int32_t vec = 1;       // elements of one load
    int32_t per = 1;       // columns: channels a thread; rows: vectors a thread
    int32_t lg = 0;        // log2 of the lanes along the points (columns) or along the row (rows)
    int32_t groups = 1;    // columns: threads along the channels; rows: rows a workgroup holds at a time
    int32_t threads = 64;
    int64_t tiles = 0;     // tiles of points or of rows
    int32_t tiles_n = 1;   // columns, vec > 1: tiles of one n
};

DISCO_HD int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- columns

struct ColPos {
    int64_t n, m;   // the first point held
    int32_t dup;    // leading elements held by another lane too (vec or more: all of them)
};

// Where lane `lane` of tile `tile` lies (vec points from m on; flat tiles, vec == 1, run over n too).
DISCO_HD ColPos col_pos(int64_t tile, int lane, int vec, int lg, int32_t tiles_n, int64_t N, int64_t M)
{
    ColPos p;
    if (vec > 1) {
        p.n = (int64_t)((uint32_t)tile / (uint32_t)tiles_n);
        const int64_t m = ((tile - p.n * tiles_n) << lg) * vec + (int64_t)lane * vec;
        p.m = m < M - vec ? m : M - vec;
        p.dup = (int32_t)(m - p.m < vec ? m - p.m : vec);
    } else {
        const int64_t q = (tile << lg) + lane, last = N * M - 1;
        const int64_t r = q < last ? q : last;
        p.n = r / M;
        p.m = r - p.n * M;
        p.dup = q > last;
    }
    return p;
}

// The tile that workgroup i of n takes so that neighbouring tiles go to one XCD (workgroups go round the 8
// XCDs): the cache lines that two tiles share are then written through one L2.
DISCO_HD int64_t xcd_tile(int64_t i, int64_t n)
{
    const int64_t q = n >> 3, r = n & 7, x = i & 7;
    return x * q + (x < r ? x : r) + (i >> 3);
}

// ---- rows

struct RowPos {
    int32_t c;      // first element held
    int32_t dup;    // leading elements held by another thread too (vec or more: all of them)
};

DISCO_HD RowPos row_pos(int v, int vec, int D)
{
    const int64_t c = (int64_t)v * vec;
    RowPos p;
    p.c = (int32_t)(c < D - vec ? c : D - vec);
    p.dup = (int32_t)(c - p.c < vec ? c - p.c : vec);
    return p;
}

// ---- geometry

constexpr int kNormMaxThreads = 1024;
constexpr int64_t kStreamBytes = (int64_t)128 << 20;  // outputs beyond these are stored past the caches: columns
constexpr int64_t kStreamRows = (int64_t)32 << 20;    // and gradients, rows and the reader (32 MiB: all XCDs' L2)
constexpr int kColsMinM = 64;    // fewer points after the axis than this: flat tiles of single elements

// A store past the L2 leaves no line there for a neighbouring tile to complete, so what is stored must be whole
// 64-byte sectors: `run` bytes a channel (columns) or a row, from aligned bases.  bf16, columns: the norm of
// 2x256x721x1440 840 against 1025 us kept in the L2; with runs that end inside a sector (1x512x361x720) 356
// against 237 us.  Between 32 and 128 MiB columns lose (2x64x360x720 39.4 against 38.5 us) and rows gain
// (20000x4096 105 against 114 us).
inline bool stream_stores(bool rows, int64_t bytes, int64_t run, const void *o0, const void *o1)
{
    return bytes > (rows ? kStreamRows : kStreamBytes) && run % 64 == 0 && (((uintptr_t)o0 | (uintptr_t)o1) & 63) == 0;
}

inline int log2_up(int64_t v)
{
    int l = 0;
    while (((int64_t)1 << l) < v) ++l;
    return l;
}

// Geometry for (N, D, M) with elements of esz bytes.  N, D, M >= 1.
inline NormGeom norm_geom(int64_t N, int64_t D, int64_t M, int esz, bool bwd)
{
    NormGeom g;
    const int vmax = 16 / esz;
    if (M == 1) {
        g.rows = 1;
        g.vec = D >= vmax ? vmax : 1;
        const int64_t nv = ceil_div64(D, g.vec);
        if (nv > (int64_t)kNormMaxThreads * 4) {
            g.loop = 1;
        } else {
            // Two vectors a thread from 9 on where there are rows for all CUs (1000000x128 8-bit 69 against 76 us);
            // a few rows are done sooner over more threads (1x256 bf16 1.9 against 2.3 us on the GPU).
            g.per = nv > (bwd ? 2048 : 512) ? 4 : nv > 32 || (nv > 8 && N >= 4096) ? 2 : 1;
            g.lg = log2_up(ceil_div64(nv, g.per));
            const int lanes = 1 << g.lg;
            g.threads = lanes > 256 ? lanes : 256;
            g.groups = g.threads / lanes;
            g.tiles = ceil_div64(N, g.groups);
            return g;
        }
    } else {
        const bool flat = M < kColsMinM;
        g.vec = flat ? 1 : vmax;
        // Channels a thread, then as many lanes along the points as the workgroup has threads for: a run of
        // 64 lanes x 16 bytes of each channel at most.  Longer runs cost memory less: forward, 2x256x721x1440 bf16,
        // 8 channels and 32 lanes 836 us, 8 and 16 860, 4 and 16 858; 8 bits, 1x80x721x1440, 8 and 64 126, 8 and 32 129,
        // 8 and 16 138.  Backward (two inputs, so half the channels fit), 2x64x361x720, 4 and 32 46.6, 4 and 16 49.6,
        // 2 and 32 52.8.
        g.per = D >= 16 && !bwd ? 8 : D >= 8 ? 4 : D >= 4 ? 2 : 1;
        const int64_t ng = ceil_div64(D, g.per);
        int lg = bwd && esz == 2 && !flat ? 5 : 6;  // the backward's LDS holds two sums a point
        while (lg < 8 && (ng << lg) < 256) ++lg;
        while (lg > 2 && (ng << lg) > kNormMaxThreads) --lg;
        // shorter runs where the points would not give every CU two tiles
        while (!flat && lg > 4 && N * ceil_div64(M, (int64_t)g.vec << lg) < 512) --lg;
        if ((ng << lg) > kNormMaxThreads) {
            g.loop = 1;
        } else {
            g.lg = lg;
            int64_t th = ng << lg;
            th = (th + 63) & ~(int64_t)63;
            g.threads = (int32_t)th;
            g.groups = (int32_t)(th >> lg);
        }
    }
    if (g.loop) {
        // one point (rows) or 32 points at a time; the threads walk the channels
        g.rows = 0;
        g.vec = 1;
        g.per = 1;
        g.lg = M == 1 ? 0 : 5;
        g.threads = kNormMaxThreads;
        g.groups = g.threads >> g.lg;
    }
    const int64_t P = ((int64_t)1 << g.lg) * g.vec;
    if (g.vec > 1) {
        g.tiles_n = (int32_t)ceil_div64(M, P);
        g.tiles = (int64_t)g.tiles_n * N;
    } else {
        g.tiles = ceil_div64(N * M, P);
    }
    return g;
}

// Columns: partial sums of one point that a workgroup joins through LDS (one a wave, or one a g where the
// lanes of a g fill whole waves).
inline int cols_parts(const NormGeom &g) { return g.threads >> (g.lg < 6 ? 6 : g.lg); }

// Dynamic LDS of the forward (ngroups: scales along the axis, 0 without an 8-bit output) and of the backward.
inline size_t norm_lds(const NormGeom &g, int ngroups)
{
    const size_t P = ((size_t)1 << g.lg) * g.vec;
    if (g.loop) return (g.groups + 1) * P * 4;
    if (g.rows) return ngroups > 1 ? (size_t)g.groups * ngroups * 4 : 0;
    return (size_t)(cols_parts(g) + 1 + ngroups) * P * 4;
}

constexpr int kBwdLdsWeights = 3;   // rows, four vectors of fp32 a thread: vectors whose weights lie in LDS

inline size_t norm_bwd_lds(const NormGeom &g, int64_t D)
{
    const size_t P = ((size_t)1 << g.lg) * g.vec;
    if (g.loop) return 2 * g.groups * P * 4;
    if (g.rows && g.per == 4 && g.vec == 4) return (size_t)kBwdLdsWeights * g.threads * 16;
    if (g.rows) return g.groups > 1 ? (size_t)g.groups * D * 8 : 0;
    const size_t join = (size_t)(2 * cols_parts(g) + 2) * P * 4;
    const size_t last = (size_t)(g.lg > 6 ? 1 << (g.lg - 6) : 1) * g.groups * g.per * 8;
    return join > last ? join : last;
}

// ---- the backward's launches

constexpr int kDwThreads = 256;

struct BwdPlan {
    NormGeom g;
    int32_t blocks = 0;    // workgroups of the first launch, each walking every blocks-th tile
    bool apart = false;    // long rows: dw is summed by a launch of its own
    int32_t parts = 0;     // rows of D partial sums of dw: one a workgroup, or one a chunk of rows
    int64_t dw_tiles = 0, dw_rows = 0;  // long rows: workgroups along the row, rows of a chunk
    // dw is written without a launch that adds the parts
    bool direct() const { return parts == 1 && (apart || !g.loop); }
    // [parts][D] fp64, then (long rows) [N] fp32 of rstd
    size_t bytes(int64_t N, int64_t D) const { return (size_t)parts * (size_t)D * 8 + (apart ? (size_t)N * 4 : 0); }
};

inline BwdPlan norm_bwd_plan(int64_t N, int64_t D, int64_t M, int esz)
{
    BwdPlan p;
    if (N == 0 || M == 0) return p;
    p.g = norm_geom(N, D, M, esz, true);
    p.apart = M == 1 && (p.g.loop || (p.g.per == 4 && esz == 2));
    // Up to two tiles are done by one workgroup, which then needs no second launch (4x617 bf16 6.4 against 10.0 us).
    const bool one = !p.g.loop && !p.apart && p.g.tiles <= 2;
    // 256 CUs; 1024 threads of these kernels' registers a CU, and half of them for rows: fewer rows open at a time
    // (259200x512 bf16 194 against 214 us, fp32 389 against 433 us).
    const int each = p.g.rows ? 512 : 1024;
    const int64_t most = one ? 1 : 256 * (p.g.threads >= each ? 1 : each / p.g.threads);
    p.blocks = (int32_t)(p.g.tiles < most ? p.g.tiles : most);
    p.parts = p.blocks;
    if (p.apart) {
        // Up to 32 rows are one chunk, which needs no third launch (9x40000 bf16 23.8 against 29.5 us); more are as many
        // chunks of 8 rows or more as 8 workgroups a CU take (40x20000 bf16 16.4 us, chunks of 32 or more 18.5).
        p.dw_tiles = ceil_div64(D, (int64_t)kDwThreads * (16 / esz));
        const int64_t want = p.dw_tiles < 2048 ? 2048 / p.dw_tiles : 1, most_parts = N <= 32 ? 1 : ceil_div64(N, 8);
        p.dw_rows = ceil_div64(N, want < most_parts ? want : most_parts);
        p.parts = (int32_t)ceil_div64(N, p.dw_rows);
    }
    return p;
}

constexpr int kDwSumThreads = 1024, kDwSumCols = 16;

// Workgroups of the launch that adds the parts of dw; longer axes are walked.
inline int64_t dw_sum_blocks(int64_t D)
{
    const int64_t all = ceil_div64(D, kDwSumCols);
    return all < (1 << 16) ? all : 1 << 16;
}

// ---- reader of the 8-bit form

constexpr int kDequantCpt = 8;   // columns: channels a thread

struct DequantGeom {
    bool vec = false;
    int32_t lg = 6;        // log2 of the lanes along the points (columns) or along the row (rows)
    int32_t chunks = 1;    // columns: workgroups along the channels
    int32_t tiles_n = 0;
    int64_t blocks = 0;    // of 256 threads
};

inline DequantGeom dequant_geom(int64_t N, int64_t D, int64_t M, int esz)
{
    const int V = 16 / esz;
    DequantGeom g;
    if (M == 1) {
        g.vec = D >= V;
        const int lg = log2_up(ceil_div64(D, g.vec ? V : 1));
        g.lg = lg < 8 ? lg : 8;
        g.blocks = ceil_div64(N, 256 >> g.lg);
    } else {
        g.vec = M >= kColsMinM;
        const int64_t P = (int64_t)64 * (g.vec ? V : 1);
        g.chunks = (int32_t)ceil_div64(D, 4 * kDequantCpt);
        g.tiles_n = g.vec ? (int32_t)ceil_div64(M, P) : 0;
        g.blocks = (g.vec ? N * g.tiles_n : ceil_div64(N * M, P)) * g.chunks;
    }
    return g;
}

}  // namespace disco
