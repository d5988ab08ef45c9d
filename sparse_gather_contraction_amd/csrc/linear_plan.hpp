// linear_plan.hpp — launch geometry and index arithmetic of the 8-bit form and the channel products (host and device).
//
// A tensor is seen as (N, D, M) around its channel axis, as the norms see it: point (n, m) is number g = n M + m,
// and its channel d lies at (n D + d) M + m.  The 8-bit form of P = N M points is (P, Dp): a point's channels lie
// together, Dp = D rounded up to 16, the places behind D hold zeros.
#pragma once

#include "norm_plan.hpp"

namespace disco {

// n / d for n < 2^31 as a product: m = ceil(2^(31 + l) / d) with l = ceil(log2 d), exact for every such n.
struct FastDiv {
    uint32_t d = 1, m = 0x80000000u, l = 0;
    DISCO_HD uint32_t div(uint32_t n) const
    {
#if defined(__HIP_DEVICE_COMPILE__)
        return __umulhi(2 * n, m) >> l;
#else
        return (uint32_t)(((uint64_t)(2 * n) * m) >> 32) >> l;
#endif
    }
};

inline FastDiv fast_div(uint32_t d)
{
    FastDiv f;
    f.d = d;
    while (((uint64_t)1 << f.l) < d) ++f.l;
    f.m = (uint32_t)((((uint64_t)1 << (31 + f.l)) + d - 1) / d);
    return f;
}

constexpr int64_t kMaxPoints = ((int64_t)1 << 31) - 4096;  // point numbers, and those a tile runs past the end, are 32 bits
constexpr int64_t kMaxChannels = 131056;                   // of a product: |sum| <= 131056 x 128 x 128 < 2^31

inline int64_t padded_channels(int64_t d) { return (d + 15) & ~(int64_t)15; }

// ---- the form's writer and reader
//
// A thread holds vectors of eight neighbouring channels.  rows: 2^lg threads a point, thread t the vectors
// t, t + lanes, ...  fields: a workgroup holds a tile of points with all their channels, thread (g, lane) the
// channels 8 g .. 8 g + 7 of the points lane*vec .. lane*vec + vec-1 (col_pos of norm_plan.hpp); the tile's
// codes pass through LDS, so that both sides of the transposition are runs.

struct FormGeom {
    int32_t rows = 0;
    int32_t loop = 0;     // 1: the channels pass the threads' registers; two passes over the data
    int32_t vec = 1;      // fields: points of one load
    int32_t per = 1;      // rows: vectors a thread
    int32_t lg = 0;       // log2 of the threads of a point (rows) or of the lanes along the points (fields)
    int32_t threads = 64;
    int32_t slots = 1;    // rows: points a workgroup holds; fields: threads along the channels
    int64_t tiles = 0;
    int32_t tiles_n = 1;  // fields, vec > 1: tiles of one n
};

constexpr int kFormChannels = 8;                 // channels of a thread's vector
// Fields: workgroups of 512 threads, two or three of them a CU, so that the loads of one run beside the turn and the stores
// of another (2x256x721x1440 bf16: writer 302 us, with 1024 threads and runs twice as long 389; reader 349 and 331;
// 80x721x1440 both 90 and 105); 1024 where that many hold the channels of a few points at least.
constexpr int kFormThreads = 512;

inline FormGeom form_geom(int64_t N, int64_t D, int64_t M, int esz)
{
    FormGeom g;
    const int64_t Dp = padded_channels(D), nv = Dp / kFormChannels;
    if (M == 1) {
        g.rows = 1;
        if (nv > 4 * (int64_t)kNormMaxThreads) {
            g.loop = 1;
        } else {
            // A wave a point up to 256 vectors, so that no join leaves the wave.
            g.per = nv > 128 ? 4 : nv > 64 ? 2 : 1;
            g.lg = log2_up(ceil_div64(nv, g.per));
            const int lanes = 1 << g.lg;
            g.threads = lanes > 256 ? lanes : 256;
            g.slots = g.threads / lanes;
            g.tiles = ceil_div64(N, g.slots);
            return g;
        }
    } else {
        const bool flat = M < kColsMinM;
        g.vec = flat ? 1 : 16 / esz;
        int lg = 6;
        while (lg < 8 && (nv << lg) < 256) ++lg;
        const int most = (nv << 2) > kFormThreads ? kNormMaxThreads : kFormThreads;
        while (lg > 2 && (nv << lg) > most) --lg;
        // shorter runs where the points would not give every CU two tiles
        while (!flat && lg > 4 && N * ceil_div64(M, (int64_t)g.vec << lg) < 512) --lg;
        if ((nv << lg) > most) {
            g.loop = 1;
        } else {
            g.lg = lg;
            g.threads = (int32_t)(((nv << lg) + 63) & ~(int64_t)63);
            g.slots = (int32_t)nv;
        }
    }
    if (g.loop) {  // one point (rows) or 32 points at a time; the threads walk the vectors
        g.vec = 1;
        g.lg = M == 1 ? 0 : 5;
        g.threads = kNormMaxThreads;
        g.slots = g.threads >> g.lg;
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

// Fields: where the codes of channels 8 g .. 8 g + 7 of the tile's point p lie in LDS.  A point's nv eights are
// turned by p / vec places, so that the lanes of a wave, which write one eight each of points vec apart, meet
// different banks.
DISCO_HD int form_lds(int p, int g, int nv, int lane_of_p)
{
    int c = g + lane_of_p % nv;
    if (c >= nv) c -= nv;
    return (p * nv + c) * 8;
}

inline size_t form_lds_bytes(const FormGeom &g, int64_t Dp)
{
    if (g.loop) return ((size_t)1 << g.lg) * 8;
    if (g.rows) return 0;
    const size_t P = ((size_t)1 << g.lg) * g.vec;
    return P * (size_t)Dp + P * 8;  // codes; two maxima a point
}

// ---- the products
//
constexpr int kFewPoints = 128;    // so many points at most: each weight is read once, 16 output channels a workgroup
constexpr int kFewWaves = 8;       // of so many waves

// Workgroups and their threads of a product, at most.
inline int64_t lin_blocks(int64_t P, int64_t Co) { return P <= kFewPoints ? ceil_div64(Co, 16) : ceil_div64(P, 128) * ceil_div64(Co, 128); }
inline int lin_threads(int64_t P) { return P <= kFewPoints ? 64 * kFewWaves : 256; }

// out[v][u] over tiles of BU x BV, u the axis that lies together in the output.  The tensor that holds the
// points may be a field: then the points' axis is cut into planes of M (plane(g) = g / M).

// The tile that workgroup i of n takes: neighbouring tiles go to one XCD (xcd_tile), u or v fastest.
DISCO_HD void lin_tile(int64_t i, int64_t n, int32_t fast, int32_t *a, int32_t *b)
{
    const int64_t t = xcd_tile(i, n);
    *b = (int32_t)(t / fast);
    *a = (int32_t)(t - (int64_t)*b * fast);
}

// LDS of a tile of rows of K bytes (64 to 1024; 8-bit channels of a step, or gradients of two bytes): slot i (16 bytes) holds row i / (K / 16), piece lin_piece(i).
// The pieces of a row are turned by the row, so that sixteen rows' equal pieces lie in sixteen different banks.
template <int K>
DISCO_HD int lin_turn(int row) { return K == 64 ? row >> 2 & 3 : K == 128 ? row >> 1 & 7 : row & 15; }
template <int K>
DISCO_HD int lin_piece(int slot) { return (slot % (K / 16)) ^ lin_turn<K>(slot / (K / 16)); }
template <int K>
DISCO_HD int lin_at(int row, int piece) { return row * K + 16 * (piece ^ lin_turn<K>(row)); }

// The weights in registers: tiles of PT points pass through a ring in LDS by direct loads, four waves of 256 threads.  A tile's
// slot i (16 bytes) holds what lin_piece says; behind it each wave's own copy of the points' scales.
//
// The product: K channels, padded.
template <int K_>
struct LStay {
    static constexpr int K = K_;
    static constexpr int PT = K == 512 ? 32 : 64;       // points of a tile
    static constexpr int RING = K >= 256 ? 3 : 4;
    static constexpr int kTile = PT * K, kStage = kTile + 4 * 256;
    static constexpr int LOADS = kTile / 16 / 256 + 1;  // direct loads of a thread and tile
};
constexpr int kStayChannels = 256;   // output channels of a workgroup

// The input's gradient.  KB: bytes of a point's gradients, padded (two an output channel).  KEPT: a checkpoint comes with them,
// between the tile and the scales.
template <int KB_, bool KEPT>
struct GStay {
    static constexpr int KB = KB_;
    static constexpr int FW = KB == 1024 ? 1 : 2;            // 32 channels each, of a wave
    static constexpr int CW = 32 * FW, CB = 4 * CW;          // channels of a wave, of a workgroup
    static constexpr int PT = KB >= 512 ? 32 : 64;           // points of a tile
    static constexpr int RING = KB == 512 || (KB <= 256 && !KEPT) ? 3 : 2;
    static constexpr int kTile = PT * KB, kKept = KEPT ? PT * CB : 0;
    static constexpr int kStage = kTile + kKept + (KEPT ? 4 * 256 : 0);
    static constexpr int LOADS = kTile / 16 / 256, KLOADS = kKept / 16 / 256;
};

// LDS of an operand staged [r][n], rows of N 16-bit elements: the 32-byte piece c of row r lies at piece
// c ^ (2 (r % 4) + r / 8 % 2).  A transposing read takes rows r .. r + 3 of two neighbouring pieces, and of rows r + 8 ..
// r + 11, at a time: these then lie in different banks.
template <int N>
DISCO_HD int bwd_across(int r, int n)
{
    const int turn = N >= 128 ? (r & 3) << 1 | ((r >> 3) & 1) : 0;   // (N = 32: four rows are 256 bytes as they lie)
    return r * N * 2 + ((((n >> 4) ^ turn) << 5) | ((n & 15) << 1));
}

// LDS of an operand staged [n][r], rows of R (64) r: the 16-byte pieces of a row are turned by the row.
template <int R>
DISCO_HD int bwd_along(int n, int piece) { return lin_at<R * 2>(n, piece); }

// The weight's gradient: the points are cut into `splits` runs of `steps` steps of 64, so that the tiles of the small
// output fill the CUs; each leaves fp32 partial sums, joined afterwards.
struct WeightPlan {
    int32_t splits = 1, steps = 1;
    int32_t nx = 1;            // tiles along C: they share a split's sums of db
};

// Tiles of the gradients: 256 x 256, 128 x 128, or for 32 input channels at most 32 of them x 256.
constexpr int kNarrow = 32;
inline bool weight_large(int64_t Co, int64_t C) { return Co > 128 && C > 128; }

inline WeightPlan weight_plan(int64_t P, int64_t C, int64_t Co)
{
    const bool large = weight_large(Co, C), narrow = C <= kNarrow;
    const int64_t bx = large ? 256 : narrow ? kNarrow : 128, ba = large || narrow ? 256 : 128;
    const int64_t tiles = ceil_div64(C, bx) * ceil_div64(Co, ba);
    const int64_t all = ceil_div64(P, 64), want = large ? 256 : 512;   // workgroups: one or two a CU
    int64_t splits = want / tiles;
    if (splits > all) splits = all;
    if (splits < 1) splits = 1;
    WeightPlan p;
    p.nx = (int32_t)ceil_div64(C, bx);
    p.steps = (int32_t)ceil_div64(all, splits);
    p.splits = (int32_t)ceil_div64(all, p.steps);
    return p;
}

inline size_t weight_bytes(const WeightPlan &p, int64_t C, int64_t Co, bool bias)
{
    return p.splits == 1 ? 0 : (size_t)p.splits * (size_t)(Co * C + (bias ? Co * p.nx : 0)) * 4;
}

}  // namespace disco
