// kernels_linear_bwd.hip — the gradients of the channel product y = x W^T + bias, whose operands are kept in 8 bits:
//
//   gx[p][c] = act'(kept[p][c]) sum_o gy[p][o] (wscale[o] w[o][c])
//   dw[o][c] = sum_p gy[p][o] (scale[p] q[p][c]),   db[o] = sum_p gy[p][o]
//
// Both are out = sum_r A(., r) X[r][.] with X[r][c] = s[r] b[r][c] an 8-bit operand whose scale belongs to the index r that
// is summed over.  The scale cannot leave the sum, so X is formed tile by tile on its way into LDS, rounded once to the data
// type (as the reader of the form would write it); the products are exact in fp32 and the sums fp32.  That one rounding of a
// term is as large as the result's own and makes its error sqrt 2 of one rounding's; 16 bits more of X would take a second
// product for each.
//
// Tile: BU x BV outputs, steps of 64 r.  X is staged [r][c] and read through the transposing LDS read.  gy comes in either
// order: with r together (rows for gx, fields for dw) it is staged [.][r] and read as it lies, else [r][.] and transposed as
// X is.  Operands pass through registers (they need converting, or lie at any element), the next step's while this one is
// multiplied; two LDS buffers.  Each part of a step is converted and put down between the products of the step before, and
// the same part of the step after it asked for at once, so that vector instructions, LDS writes and loads run beside the
// matrix cores (8192^3 bf16 1.02 PFLOP/s; 259200 points 512 to 2048 0.84; all at a step's end: 0.78).  Large outputs are
// bound by the matrix cores and these together, outputs of one tile (256 x 256 at 2076480 points: 409 us, 3.9 TB/s) by the one
// step of loads that the registers leave room for.
#include <algorithm>
#include <type_traits>

#include "act_device.hpp"
#include "kernels.hpp"
#include "linear.hpp"
#include "linear_device.hpp"

namespace disco {

namespace {

enum Mode { kInRows, kInField, kWeightRows, kWeightField };

template <int BU_, int BV_, int WU_, int WV_, int R_>
struct BTile {
    static constexpr int BU = BU_, BV = BV_, WU = WU_, WV = WV_;
    static constexpr int R = R_;                                 // r of a step
    static constexpr int kThreads = 64 * WU * WV;
    static constexpr int FU = BU / WU / 32, FV = BV / WV / 32;
    static constexpr int kStage = (BU + BV) * R * 2;
};
typedef BTile<256, 256, 2, 4, 64> BLarge;
typedef BTile<128, 128, 2, 2, 64> BSmall;
typedef BTile<32, 256, 1, 4, 64> BNarrowU;   // few input channels, X along u
typedef BTile<256, 32, 4, 1, 64> BNarrowV;   // and along v

struct BwdArgs {
    const uint16_t *gy;
    const int8_t *q;
    const float *scale;
    const int8_t *kept;
    const float *kept_scale;
    void *out;
    void *db;
    float *ws, *ws_db;             // weight with more than one split
    Planes pl, out_pl;             // gy's points or rows, and the output's
    uint32_t A, X, R;              // sizes of gy's free axis, of X's (C) and of the summed one
    int32_t nt;                    // input: stores past the caches
    int32_t Cp, na, nx, splits, steps;  // tiles; steps of a split
};

// The matrix cores' operand: 32 rows n0 .., lane n0 + lane % 32 holding r = r0 + 8 (lane / 32) .. + 7.
template <int N>
__device__ __forceinline__ bf16x8 frag_across(const unsigned char *op, int n0, int r0, int lane)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef s16x4 __attribute__((address_space(3))) *ptr;
    // 16 lanes read four rows of 16 elements, each lane a quarter of a row, and get a column each
    const int n = n0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3), r = r0 + 8 * (lane >> 5) + ((lane >> 2) & 3);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(op + bwd_across<N>(r, n)));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(op + bwd_across<N>(r + 4, n)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int R>
__device__ __forceinline__ bf16x8 frag_along(const unsigned char *op, int n0, int r0, int lane)
{
    return *reinterpret_cast<const bf16x8 *>(op + bwd_along<R>(n0 + (lane & 31), (r0 >> 3) + (lane >> 5)));
}

// Sixteen 8-bit values times a scale, to 16 bits.
template <bool F16>
__device__ __forceinline__ void form16(const u32x4 &w, float s, u32x4 &lo, u32x4 &hi)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t d = w[i >> 1];
        const int sh = 16 * (i & 1);
        const uint32_t v = pack2<F16>((float)(int8_t)(d >> sh) * s, (float)(int8_t)(d >> (sh + 8)) * s);
        if (i < 4) lo[i] = v;
        else hi[i - 4] = v;
    }
}

template <typename L, bool F16, int MODE, int ACT, bool DB>
__global__ __launch_bounds__(L::kThreads, 2) void linear_bwd_kernel(BwdArgs a)
{
    typedef typename std::conditional<F16, f16_t, bf16_t>::type T;
    constexpr bool kWeight = MODE == kWeightRows || MODE == kWeightField;
    constexpr bool kAlong = MODE == kInRows || MODE == kWeightField;         // gy's r lie together
    constexpr bool kPlanes = MODE == kInField || MODE == kWeightField;
    constexpr bool XU = MODE != kInField;                                    // X's axis lies together in the output
    constexpr int BA = XU ? L::BV : L::BU, BX = XU ? L::BU : L::BV;          // the tile along gy's axis and X's
    constexpr int FU = L::FU, FV = L::FV;
    constexpr int LA = BA * L::R / 8 / L::kThreads, LX = (BX * L::R / 16 + L::kThreads - 1) / L::kThreads;
    constexpr bool kXAll = BX * L::R / 16 % L::kThreads == 0;                // else the first threads have a piece of X
    constexpr int kA = BA * L::R * 2;
    // outputs: staged in fp32 where a factor follows (rows), or for the partial sums
    constexpr bool kFieldFactor = MODE == kInField && ACT != DISCO_ACT_NONE;
    constexpr int kTurn = 32 * (128 + 16) * L::WU * L::WV;          // kFieldFactor: LDS of the waves' pieces, then
    constexpr int KN = L::BU * L::BV / 16 / L::kThreads;            // the checkpoint [BU][BV + 16], its scales [BU]
    static_assert(!kFieldFactor || kTurn + L::BU * (L::BV + 16 + 4) <= 2 * L::kStage, "the checkpoint's tile fits the buffers");
    constexpr bool kFactor = MODE == kInRows && ACT != DISCO_ACT_NONE;
    __shared__ __attribute__((aligned(16))) unsigned char smem[2 * L::kStage];

    int ta, tx, z = 0;
    int64_t tile = xcd_tile(blockIdx.x, (int64_t)a.na * a.nx * a.splits);
    if (kWeight) {  // the tiles of one split follow each other: they read the same points
        z = (int)(tile / (a.na * a.nx));
        tile -= (int64_t)z * a.na * a.nx;
        ta = (int)(tile / a.nx);
        tx = (int)(tile - (int64_t)ta * a.nx);
    } else {        // the tiles of the same points
        ta = (int)(tile / a.nx);
        tx = (int)(tile - (int64_t)ta * a.nx);
    }
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wu = wave % L::WU, wv = wave / L::WU;
    const uint32_t a0 = (uint32_t)ta * BA, x0 = (uint32_t)tx * BX;
    const uint32_t r_begin = kWeight ? (uint32_t)z * (uint32_t)a.steps * L::R : 0u;
    const uint32_t r_left = a.R - r_begin;
    const int nk = (int)((kWeight && r_left > (uint32_t)a.steps * L::R) ? a.steps : (r_left + L::R - 1) / L::R);

    // db: wave wu < FV sums the gradients of its columns' piece wu, or a wave alone along u all of them
    static_assert(!DB || FV <= L::WU || L::WU == 1, "a wave for each piece");
    constexpr int DBN = DB && FV > L::WU ? FV : 1;
    f32x16 d[FU][FV], dbs[DBN];
#pragma unroll
    for (int i = 0; i < FU; ++i)
#pragma unroll
        for (int j = 0; j < FV; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) d[i][j][e] = 0.0f;
#pragma unroll
    for (int n = 0; n < DBN; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) dbs[n][e] = 0.0f;
    // db: the tiles of one split and gy's tile share its steps (step t is tile t % shares), so that none is slower
    const int db_shares = DB && a.splits > 1 ? a.nx : 1;
    int db_turn = tx < db_shares ? tx : -1;   // steps until this tile's next share; -1: none

    u32x4 pa[LA], px[LX];
    float ps[LX];
    // Where this thread's pieces lie: A's piece i is row an + i kAR (r together) or r ar + i kAR (else); X's row xr + i kXR.
    constexpr int kAR = kAlong ? L::kThreads / (L::R / 8) : L::kThreads / (BA / 8), kXR = L::kThreads / (BX / 16);
    const int ar = kAlong ? 8 * (tid % (L::R / 8)) : tid / (BA / 8), an = kAlong ? tid / (L::R / 8) : 8 * (tid % (BA / 8));
    const int xr = tid / (BX / 16), xn = 16 * (tid % (BX / 16));
    const bool has_x = kXAll || xr < L::R;
    const int64_t a_stride = a.pl.template stride<kPlanes>();
    const uint16_t *a_run = a.gy + (kAlong ? (int64_t)(a0 + an) * a_stride : a.pl.template run<kPlanes>(a0 + an < a.A ? a0 + an : 0));
    const int8_t *x_run = a.q + x0 + xn;
    // whether a step's pieces are all there and whole: then they are loaded as they lie, else one by one
    const bool n_full = a0 + BA <= a.A && x0 + BX <= (uint32_t)a.Cp &&
                        (kAlong || !kPlanes || a0 - a.pl.by_m.div(a0) * (uint32_t)a.pl.M + BA <= (uint32_t)a.pl.M);
    auto step_full = [&](int t) {
        const uint32_t r0 = r_begin + (uint32_t)t * L::R;
        return n_full && r0 + L::R <= a.R && (!kAlong || !kPlanes || r0 - a.pl.by_m.div(r0) * (uint32_t)a.pl.M + L::R <= (uint32_t)a.pl.M);
    };
    auto at_a = [&](int t) {
        const uint32_t r0 = r_begin + (uint32_t)t * L::R;
        return kAlong ? a_run + a.pl.template run<kPlanes>(r0 + ar) : a_run + (int64_t)(r0 + ar) * a_stride;
    };
    auto load_a = [&](const uint16_t *p, int i) { pa[i] = load_as<false, u32x4>(p + (int64_t)i * kAR * a_stride); };
    auto load_x = [&](uint32_t r, int i) {
        if (!has_x) return;
        px[i] = *(const u32x4 *)(x_run + (int64_t)(r + i * kXR) * a.Cp);
        ps[i] = a.scale[r + i * kXR];
    };
    auto fetch = [&](int t) {
        const uint32_t r0 = r_begin + (uint32_t)t * L::R;
        if (step_full(t)) {
            const uint16_t *p = at_a(t);
#pragma unroll
            for (int i = 0; i < LA; ++i) load_a(p, i);
#pragma unroll
            for (int i = 0; i < LX; ++i) load_x(r0 + xr, i);
            return;
        }
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const uint32_t r = r0 + ar + (kAlong ? 0 : i * kAR), n = a0 + an + (kAlong ? i * kAR : 0);
            if constexpr (kAlong) pa[i] = n < a.A ? load_run<kPlanes>(a.gy, a.pl, n, r, a.R) : u32x4{0, 0, 0, 0};
            else pa[i] = r < a.R ? load_run<kPlanes>(a.gy, a.pl, r, n, a.A) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            const uint32_t r = r0 + xr + i * kXR, c = x0 + xn;
            const bool in = r < a.R && has_x;
            px[i] = in && c < (uint32_t)a.Cp ? *(const u32x4 *)(a.q + (int64_t)r * a.Cp + c) : u32x4{0, 0, 0, 0};
            ps[i] = in ? a.scale[r] : 0.0f;
        }
    };
    auto stage_a = [&](unsigned char *buf, int i) {
        if constexpr (kAlong) *(u32x4 *)(buf + bwd_along<L::R>(an + i * kAR, tid % (L::R / 8))) = pa[i];
        else *(u32x4 *)(buf + bwd_across<BA>(ar + i * kAR, an)) = pa[i];
    };
    auto stage_x = [&](unsigned char *buf, int i) {
        if (!has_x) return;
        u32x4 lo, hi;
        form16<F16>(px[i], ps[i], lo, hi);
        unsigned char *to = buf + kA + bwd_across<BX>(xr + i * kXR, xn);
        // every other eight lanes the second half first: sixteen lanes then meet all banks
        const int turn = (tid >> 3) & 1;
        *(u32x4 *)(to + 16 * turn) = turn ? hi : lo;
        *(u32x4 *)(to + 16 - 16 * turn) = turn ? lo : hi;
    };
    // the parts of a step, X's before A's, are put down behind its products ks = 1 ..
    constexpr int NKS = L::R / 16;
    auto part_of = [](int q) { return q * (NKS - 1) / (LX + LA) + 1; };
    fetch(0);
#pragma unroll
    for (int i = 0; i < LA; ++i) stage_a(smem, i);
#pragma unroll
    for (int i = 0; i < LX; ++i) stage_x(smem, i);
    if (nk > 1) fetch(1);
    __syncthreads();
    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = __builtin_bit_cast(__bf16, (uint16_t)(F16 ? 0x3c00 : 0x3f80));
    for (int t = 0; t < nk; ++t) {
        const unsigned char *cur = smem + (t & 1) * L::kStage;
        unsigned char *next = smem + ((t + 1) & 1) * L::kStage;
        // the step after the next, whole: its pieces are asked for where the next step's leave their registers
        const bool ahead = t + 2 < nk && step_full(t + 2);
        const uint16_t *pa2 = at_a(t + 2);
        const uint32_t xr2 = r_begin + (uint32_t)(t + 2) * L::R + xr;
#pragma unroll
        for (int ks = 0; ks < L::R / 16; ++ks) {
            bf16x8 fu[FU], fv[FV];
            auto of_a = [&](int n0) {
                if constexpr (kAlong) return frag_along<L::R>(cur, n0, 16 * ks, lane);
                else return frag_across<BA>(cur, n0, 16 * ks, lane);
            };
            auto of_x = [&](int n0) { return frag_across<BX>(cur + kA, n0, 16 * ks, lane); };
#pragma unroll
            for (int i = 0; i < FU; ++i) fu[i] = XU ? of_x(L::BU / L::WU * wu + 32 * i) : of_a(L::BU / L::WU * wu + 32 * i);
#pragma unroll
            for (int j = 0; j < FV; ++j) fv[j] = XU ? of_a(L::BV / L::WV * wv + 32 * j) : of_x(L::BV / L::WV * wv + 32 * j);
#pragma unroll
            for (int i = 0; i < FU; ++i)
#pragma unroll
                for (int j = 0; j < FV; ++j) d[i][j] = bwd_mma<F16>(fu[i], fv[j], d[i][j]);
            if constexpr (DB) {
                if (db_turn == 0 && wu < FV)
#pragma unroll
                    for (int n = 0; n < DBN; ++n)
                        dbs[n] = bwd_mma<F16>(ones, DBN > 1 ? fv[n] : wu == 0 ? fv[0] : fv[FV - 1], dbs[n]);
            }
            // the next step's operands, asked for a step ago, into the other buffer between the products (behind the last
            // step nothing reads them)
#pragma unroll
            for (int i = 0; i < LX; ++i)
                if (part_of(i) == ks) {
                    stage_x(next, i);
                    if (ahead) load_x(xr2, i);
                }
#pragma unroll
            for (int i = 0; i < LA; ++i)
                if (part_of(LX + i) == ks) {
                    stage_a(next, i);
                    if (ahead) load_a(pa2, i);
                }
        }
        if constexpr (DB) db_turn = db_turn == 0 ? db_shares - 1 : db_turn - 1;
        if (t + 2 < nk && !ahead) fetch(t + 2);
        // the other buffer is whole, and this one is read; loads in flight stay there
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        bare_barrier();
    }
    __syncthreads();

    // A lane holds column v = lane % 32 and rows u = 8 (e / 4) + 4 (lane / 32) + e % 4 of each accumulator.
    const int r = lane & 31, h = lane >> 5;
    const uint32_t U = XU ? a.X : a.A, V = XU ? a.A : a.X;
    const uint32_t uw = (XU ? x0 : a0) + L::BU / L::WU * wu, vw = (XU ? a0 : x0) + L::BV / L::WV * wv;
    if constexpr (DB) {
        if (tx < db_shares && wu < FV && h == 0)
#pragma unroll
            for (int n = 0; n < DBN; ++n) {
                const uint32_t o = vw + 32 * (DBN > 1 ? n : wu) + r;
                if (o < a.A) {
                    if (a.splits > 1) a.ws_db[((int64_t)z * a.nx + tx) * a.A + o] = dbs[n][0];
                    else store_elem((T *)a.db, o, dbs[n][0]);
                }
            }
    }
    unsigned char *ktile = smem + kTurn;
    float *kscale = (float *)(ktile + L::BU * (L::BV + 16));
    if constexpr (kFieldFactor) {   // the checkpoint's tile (points a0 .., channels x0 ..) to LDS
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int s = i * L::kThreads + tid, row = s / (L::BV / 16), c = 16 * (s % (L::BV / 16));
            const uint32_t pt = a0 + row < U ? a0 + row : U - 1;
            const u32x4 w = x0 + c < (uint32_t)a.Cp ? *(const u32x4 *)(a.kept + (int64_t)pt * a.Cp + x0 + c) : u32x4{0, 0, 0, 0};
            *(u32x4 *)(ktile + row * (L::BV + 16) + c) = w;
        }
        for (int i = tid; i < L::BU; i += L::kThreads) kscale[i] = a.kept_scale[a0 + i < U ? a0 + i : U - 1];
        __syncthreads();
    }
    // Each wave turns 32 v x UR u at a time in LDS of its own, and writes them as runs along u.
    auto each = [&](auto fp32) {
        constexpr bool kF32 = decltype(fp32)::value;
        typedef typename std::conditional<kF32, float, T>::type S;   // as staged
        constexpr int ES = (int)sizeof(S);
        constexpr int ROW = kFieldFactor ? 128 : 256;
        constexpr int UR = FU * 32 * ES > ROW ? ROW / ES : FU * 32, FP = UR / 32, PITCH = UR * ES + 16;
        constexpr int LEN = kFactor ? 8 : 16 / ES, PIECES = UR / LEN;   // values of a lane's run, runs of a row
        static_assert(32 * PITCH * L::WU * L::WV <= 2 * L::kStage, "the pieces fit the buffers");
        typedef typename std::conditional<kF32 && !kFactor, float, T>::type O;
        O *base = (O *)a.out;
        if constexpr (kF32 && !kFactor) base = a.ws + (int64_t)z * V * U;
        unsigned char *st = smem + wave * 32 * PITCH;
        constexpr int ROWS = 32 * PIECES / 64;   // a lane's runs of a piece
        // kFactor (u: channels, v: points): the checkpoint of a lane's runs, asked for before the piece is turned
        u32x2 kept[kFactor ? ROWS : 1];
        float ks[kFactor ? ROWS : 1];
#pragma unroll
        for (int p = 0; p < FU / FP; ++p) {
            const uint32_t ul = uw + UR * p + lane % PIECES * LEN;
            const RunOut<O, MODE == kInField> out(base, a.out_pl, ul, U);
#pragma unroll
            for (int j = 0; j < FV; ++j) {
                if constexpr (kFactor) {
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        const uint32_t v = vw + 32 * j + i * (64 / PIECES) + lane / PIECES, at = v < V ? v : V - 1;
                        kept[i] = *(const u32x2 *)(a.kept + (int64_t)at * a.Cp + (ul < U ? ul : 0));
                        ks[i] = a.kept_scale[at];
                    }
                }
#pragma unroll
                for (int i = 0; i < FP; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int ur = 32 * i + 8 * g + 4 * h;
                        f32x4 f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = d[FP * p + i][j][4 * g + e];
                        if constexpr (kFieldFactor) {  // u: points, v: channels
                            const int at = L::BU / L::WU * wu + UR * p + ur;
                            const f32x4 ksc = *(const f32x4 *)&kscale[at];
                            const unsigned char *kb = ktile + at * (L::BV + 16) + L::BV / L::WV * wv + 32 * j + r;
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[e] *= act_slope<ACT>((float)(int8_t)kb[e * (L::BV + 16)] * ksc[e]);
                        }
                        put4<S>(st + r * PITCH + ur * ES, f);
                    }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    const int row = i * (64 / PIECES) + lane / PIECES;
                    const uint32_t v = vw + 32 * j + row;
                    if constexpr (kFactor) {  // u: channels, v: points; eight channels a lane
                        const unsigned char *from = st + row * PITCH + lane % PIECES * 32;
                        const f32x4 x = *(const f32x4 *)from, y = *(const f32x4 *)(from + 16);
                        if (v >= V || ul >= U) continue;
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = (e < 4 ? x[e & 3] : y[e & 3]) * act_slope<ACT>((float)(int8_t)(kept[i][e / 4] >> (8 * (e % 4))) * ks[i]);
                        out.put(v, u32x4{pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7])}, a.nt);
                    } else {
                        const u32x4 w = *(const u32x4 *)(st + row * PITCH + lane % PIECES * 16);
                        if (v < V) out.put(v, w, !kWeight && a.nt);
                    }
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
        }
    };
    if constexpr (kFactor) each(std::true_type());
    else if (kWeight && a.splits > 1) each(std::true_type());
    else each(std::false_type());
}

// out = the sum over the splits of their partial sums, four neighbouring values a thread: 16 fours x 16 runs of splits a
// workgroup, joined in LDS in a fixed order.  The workgroups behind the first `blocks` join db.
struct JoinArgs {
    const float *ws, *ws_db;
    void *out, *db;
    int64_t n, n_db, blocks;
    int32_t splits, splits_db;
};

template <typename T>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a)
{
    __shared__ double part[16][16][4];
    const bool db = blockIdx.x >= a.blocks;
    const float *ws = db ? a.ws_db : a.ws;
    const int64_t n = db ? a.n_db : a.n;
    const int splits = db ? a.splits_db : a.splits;
    const int t = threadIdx.x, x = t & 15, y = t >> 4;
    const int64_t i = ((blockIdx.x - (db ? a.blocks : 0)) * 16 + x) * 4;
    double s[4] = {0, 0, 0, 0};
    const int each = (splits + 15) / 16, z1 = min(splits, (y + 1) * each);
    if (i + 4 <= n) {
#pragma unroll 8
        for (int z = y * each; z < z1; ++z) {
            const f32x4 v = load_as<false, f32x4>(ws + (int64_t)z * n + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += v[e];
        }
    } else {
        for (int z = y * each; z < z1; ++z)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n) s[e] += ws[(int64_t)z * n + i + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[y][x][e] = s[e];
    __syncthreads();
    if (y < 4 && i + y < n) {
        double v = 0;
        for (int k = 0; k < 16; ++k) v += part[k][x][y];
        store_elem((T *)(db ? a.db : a.out), i + y, (float)v);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void zero_kernel(T *out, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) store_elem(out, i, 0.0f);
}

BwdArgs bwd_args(const LinearBwdLaunch &l)
{
    BwdArgs a;
    a.gy = (const uint16_t *)l.gy; a.q = l.q; a.scale = l.scale; a.kept = l.kept; a.kept_scale = l.kept_scale;
    a.out = l.out; a.db = l.db; a.ws = l.workspace;
    a.ws_db = l.workspace ? l.workspace + (int64_t)l.splits * l.Co * l.C : nullptr;
    a.pl.by_m = fast_div((uint32_t)l.M); a.pl.M = l.M; a.pl.J = l.Co; a.pl.ld = l.Co;
    a.out_pl = a.pl; a.out_pl.J = l.C; a.out_pl.ld = l.C;   // gx's points or rows, or the rows of dw
    a.X = (uint32_t)l.C; a.Cp = (int32_t)l.Cp;
    a.splits = 1; a.steps = 0;
    // (259200 rows, 2048 from 512: 817 -> 773 us)
    a.nt = stream_stores(l.M == 1, l.P * l.C * 2, (l.M == 1 ? l.C : l.M) * 2, l.out, nullptr);
    return a;
}

template <typename L, bool F16, int MODE, int ACT, bool DB>
hipError_t launch_mode(BwdArgs a, hipStream_t s)
{
    constexpr int BA = MODE == kInField ? L::BU : L::BV, BX = MODE == kInField ? L::BV : L::BU;
    a.na = (int32_t)(((int64_t)a.A + BA - 1) / BA);
    a.nx = (int32_t)(((int64_t)a.X + BX - 1) / BX);
    linear_bwd_kernel<L, F16, MODE, ACT, DB><<<dim3((uint32_t)(a.na * a.nx * a.splits)), dim3(L::kThreads), 0, s>>>(a);
    return hipGetLastError();
}

// 256 x 256 where the channels fill it and every CU has one (259200 rows, 2048 to 512: 694 us against 883; 1000 rows of 1024:
// 37 against 25).
template <bool F16, int MODE, int ACT>
hipError_t input_tiles(const BwdArgs &a, hipStream_t s)
{
    if (a.X > 128 && ceil_div64(a.A, 256) * ceil_div64(a.X, 256) >= 256) return launch_mode<BLarge, F16, MODE, ACT, false>(a, s);
    if (a.X <= kNarrow) return launch_mode<typename std::conditional<MODE == kInField, BNarrowV, BNarrowU>::type, F16, MODE, ACT, false>(a, s);
    return launch_mode<BSmall, F16, MODE, ACT, false>(a, s);
}

template <bool F16, int MODE>
hipError_t input_act(const LinearBwdLaunch &l, const BwdArgs &a, hipStream_t s)
{
    return l.act == DISCO_ACT_GELU ? input_tiles<F16, MODE, DISCO_ACT_GELU>(a, s)
         : l.act == DISCO_ACT_SILU ? input_tiles<F16, MODE, DISCO_ACT_SILU>(a, s)
                                   : input_tiles<F16, MODE, DISCO_ACT_NONE>(a, s);
}

template <bool F16>
hipError_t input_typed(const LinearBwdLaunch &l, hipStream_t s)
{
    BwdArgs a = bwd_args(l);
    a.A = (uint32_t)l.P;
    a.R = (uint32_t)l.Co;
    if (bwd_stays(l)) return launch_linear_bwd_stay(l, a.nt != 0, s);
    return l.M > 1 ? input_act<F16, kInField>(l, a, s) : input_act<F16, kInRows>(l, a, s);
}

template <bool F16, int MODE>
hipError_t weight_tiles(const LinearBwdLaunch &l, const BwdArgs &a, hipStream_t s)
{
    if (weight_large(l.Co, l.C))
        return l.db ? launch_mode<BLarge, F16, MODE, DISCO_ACT_NONE, true>(a, s) : launch_mode<BLarge, F16, MODE, DISCO_ACT_NONE, false>(a, s);
    if (l.C <= kNarrow)
        return l.db ? launch_mode<BNarrowU, F16, MODE, DISCO_ACT_NONE, true>(a, s) : launch_mode<BNarrowU, F16, MODE, DISCO_ACT_NONE, false>(a, s);
    return l.db ? launch_mode<BSmall, F16, MODE, DISCO_ACT_NONE, true>(a, s) : launch_mode<BSmall, F16, MODE, DISCO_ACT_NONE, false>(a, s);
}

template <bool F16>
hipError_t weight_typed(const LinearBwdLaunch &l, hipStream_t s)
{
    typedef typename std::conditional<F16, f16_t, bf16_t>::type T;
    if (l.P == 0) {
        const int64_t n = l.Co * l.C;
        zero_kernel<T><<<dim3((uint32_t)std::min<int64_t>(ceil_div64(n, 256), 4096)), dim3(256), 0, s>>>((T *)l.out, n);
        if (l.db) zero_kernel<T><<<dim3((uint32_t)std::min<int64_t>(ceil_div64(l.Co, 256), 4096)), dim3(256), 0, s>>>((T *)l.db, l.Co);
        return hipGetLastError();
    }
    BwdArgs a = bwd_args(l);
    a.A = (uint32_t)l.Co;
    a.R = (uint32_t)l.P;
    const WeightPlan p = weight_plan(l.P, l.C, l.Co);
    a.splits = p.splits;
    a.steps = p.steps;
    hipError_t e = l.M > 1 ? weight_tiles<F16, kWeightField>(l, a, s) : weight_tiles<F16, kWeightRows>(l, a, s);
    if (e != hipSuccess || p.splits == 1) return e;
    JoinArgs j;
    j.ws = a.ws; j.ws_db = a.ws_db; j.out = l.out; j.db = l.db;
    j.n = l.Co * l.C; j.n_db = l.db ? l.Co : 0;
    j.blocks = ceil_div64(j.n, 64);
    j.splits = p.splits; j.splits_db = p.splits * p.nx;
    join_kernel<T><<<dim3((uint32_t)(j.blocks + ceil_div64(j.n_db, 64))), dim3(256), 0, s>>>(j);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_bwd_input(const LinearBwdLaunch &l, hipStream_t s)
{
    return l.dtype == 2 ? input_typed<true>(l, s) : input_typed<false>(l, s);
}

hipError_t launch_linear_bwd_weight(const LinearBwdLaunch &l, hipStream_t s)
{
    return l.dtype == 2 ? weight_typed<true>(l, s) : weight_typed<false>(l, s);
}

}  // namespace disco
