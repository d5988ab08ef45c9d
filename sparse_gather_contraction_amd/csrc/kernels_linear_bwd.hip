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
// multiplied; two LDS buffers.
#include <algorithm>
#include <type_traits>

#include "act_device.hpp"
#include "kernels.hpp"
#include "linear.hpp"
#include "linear_device.hpp"

namespace disco {

namespace {

enum Mode { kInRows, kInField, kWeightRows, kWeightField };

template <int BU_, int BV_, int WU_, int WV_>
struct BTile {
    static constexpr int BU = BU_, BV = BV_, WU = WU_, WV = WV_;
    static constexpr int kThreads = 64 * WU * WV;
    static constexpr int FU = BU / WU / 32, FV = BV / WV / 32;
    static constexpr int kStage = (BU + BV) * kBR * 2;
};
typedef BTile<256, 256, 2, 4> BLarge;
typedef BTile<128, 128, 2, 2> BSmall;

struct BwdArgs {
    const uint16_t *gy;
    const int8_t *q;
    const float *scale;
    const int8_t *kept;
    const float *kept_scale;
    void *out;
    void *db;
    float *ws, *ws_db;             // weight with more than one split
    Planes pl;                     // the points of gy (and of gx)
    int64_t ld;                    // rows of gy
    uint32_t A, X, R;              // sizes of gy's free axis, of X's (C) and of the summed one
    int32_t Cp, na, nx, splits, steps;  // tiles; steps of a split
};

template <bool F16>
__device__ __forceinline__ f32x16 bwd_mma(bf16x8 a, bf16x8 b, f32x16 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

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
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ bf16x8 frag_along(const unsigned char *op, int n0, int r0, int lane)
{
    return *reinterpret_cast<const bf16x8 *>(op + bwd_along(n0 + (lane & 31), (r0 >> 3) + (lane >> 5)));
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
__global__ __launch_bounds__(L::kThreads) void linear_bwd_kernel(BwdArgs a)
{
    typedef typename std::conditional<F16, f16_t, bf16_t>::type T;
    constexpr bool kWeight = MODE == kWeightRows || MODE == kWeightField;
    constexpr bool kAlong = MODE == kInRows || MODE == kWeightField;         // gy's r lie together
    constexpr bool kPlanes = MODE == kInField || MODE == kWeightField;
    constexpr bool XU = MODE != kInField;                                    // X's axis lies together in the output
    constexpr int BA = XU ? L::BV : L::BU, BX = XU ? L::BU : L::BV;          // the tile along gy's axis and X's
    constexpr int FU = L::FU, FV = L::FV;
    constexpr int LA = BA * kBR / 8 / L::kThreads, LX = BX * kBR / 16 / L::kThreads;
    constexpr int kA = BA * kBR * 2;
    // outputs: staged in fp32 where a factor follows (rows), or for the partial sums
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
    const uint32_t r_begin = kWeight ? (uint32_t)z * (uint32_t)a.steps * kBR : 0u;
    const uint32_t r_left = a.R - r_begin;
    const int nk = (int)((kWeight && r_left > (uint32_t)a.steps * kBR) ? a.steps : (r_left + kBR - 1) / kBR);

    f32x16 d[FU][FV], dbs;
#pragma unroll
    for (int i = 0; i < FU; ++i)
#pragma unroll
        for (int j = 0; j < FV; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) d[i][j][e] = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) dbs[e] = 0.0f;
    const bool has_db = DB && tx == 0;

    u32x4 pa[LA], px[LX];
    float ps[LX];
    auto fetch = [&](int t) {
        const uint32_t r0 = r_begin + (uint32_t)t * kBR;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int s = i * L::kThreads + tid;
            if constexpr (kAlong) {
                const uint32_t n = a0 + (s >> 3), r = r0 + 8 * (s & 7);
                pa[i] = n < a.A ? load_run<kPlanes>(a.gy, a.pl, a.ld, n, r, a.R) : u32x4{0, 0, 0, 0};
            } else {
                const uint32_t r = r0 + s / (BA / 8), n = a0 + 8 * (s % (BA / 8));
                pa[i] = r < a.R ? load_run<kPlanes>(a.gy, a.pl, a.ld, r, n, a.A) : u32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            const int s = i * L::kThreads + tid;
            const uint32_t r = r0 + s / (BX / 16), c = x0 + 16 * (s % (BX / 16));
            const bool in = r < a.R;
            px[i] = in && c < (uint32_t)a.Cp ? *(const u32x4 *)(a.q + (int64_t)r * a.Cp + c) : u32x4{0, 0, 0, 0};
            ps[i] = in ? a.scale[r] : 0.0f;
        }
    };
    auto stage = [&](unsigned char *buf) {
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int s = i * L::kThreads + tid;
            if constexpr (kAlong) *(u32x4 *)(buf + bwd_along(s >> 3, s & 7)) = pa[i];
            else *(u32x4 *)(buf + bwd_across<BA>(s / (BA / 8), 8 * (s % (BA / 8)))) = pa[i];
        }
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            const int s = i * L::kThreads + tid;
            u32x4 lo, hi;
            form16<F16>(px[i], ps[i], lo, hi);
            unsigned char *to = buf + kA + bwd_across<BX>(s / (BX / 16), 16 * (s % (BX / 16)));
            *(u32x4 *)to = lo;
            *(u32x4 *)(to + 16) = hi;
        }
    };
    fetch(0);
    stage(smem);
    __syncthreads();
    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = __builtin_bit_cast(__bf16, (uint16_t)(F16 ? 0x3c00 : 0x3f80));
    for (int t = 0; t < nk; ++t) {
        const unsigned char *cur = smem + (t & 1) * L::kStage;
        if (t + 1 < nk) fetch(t + 1);
#pragma unroll
        for (int ks = 0; ks < kBR / 16; ++ks) {
            bf16x8 fu[FU], fv[FV];
            auto of_a = [&](int n0) {
                if constexpr (kAlong) return frag_along(cur, n0, 16 * ks, lane);
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
            // db: wave wu < FV sums the gradients of its columns' piece wu
            if constexpr (DB) {
                static_assert(!DB || L::FV <= L::WU, "a wave for each piece");
                if (has_db && wu < FV) dbs = bwd_mma<F16>(ones, wu == 0 ? fv[0] : fv[FV - 1], dbs);
            }
        }
        if (t + 1 < nk) stage(smem + ((t + 1) & 1) * L::kStage);
        __syncthreads();
    }

    // A lane holds column v = lane % 32 and rows u = 8 (e / 4) + 4 (lane / 32) + e % 4 of each accumulator.
    const int r = lane & 31, h = lane >> 5;
    const uint32_t U = XU ? a.X : a.A, V = XU ? a.A : a.X;
    const uint32_t uw = (XU ? x0 : a0) + L::BU / L::WU * wu, vw = (XU ? a0 : x0) + L::BV / L::WV * wv;
    if constexpr (DB) {
        if (has_db && wu < FV && h == 0) {
            const uint32_t o = vw + 32 * wu + r;
            if (o < a.A) {
                if (a.splits > 1) a.ws_db[(int64_t)z * a.A + o] = dbs[0];
                else store_elem((T *)a.db, o, dbs[0]);
            }
        }
    }
    auto each = [&](auto fp32) {
        constexpr bool kF32 = decltype(fp32)::value;
        constexpr int ES = kF32 ? 4 : 2;
        constexpr int UR = FU * 32 * ES > 256 ? 256 / ES : FU * 32, FP = UR / 32, PITCH = UR * ES + 16, PIECES = UR * ES / 16;
        static_assert(32 * PITCH * L::WU * L::WV <= 2 * L::kStage, "the pieces fit the buffers");
        unsigned char *st = smem + wave * 32 * PITCH;
#pragma unroll
        for (int j = 0; j < FV; ++j)
#pragma unroll
            for (int p = 0; p < FU / FP; ++p) {
#pragma unroll
                for (int i = 0; i < FP; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int ur = 32 * i + 8 * g + 4 * h;
                        float f[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = d[FP * p + i][j][4 * g + e];
                        if constexpr (MODE == kInField && ACT != DISCO_ACT_NONE) {  // u: points, v: channels
                            const uint32_t c = vw + 32 * j + r;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t pt = uw + UR * p + ur + e, at = pt < U ? pt : U - 1;
                                const int k = a.kept[(int64_t)at * a.Cp + (c < V ? c : V - 1)];
                                f[e] *= act_slope<ACT>((float)k * a.kept_scale[at]);
                            }
                        }
                        unsigned char *to = st + r * PITCH + ur * ES;
                        if constexpr (kF32) *(f32x4 *)to = f32x4{f[0], f[1], f[2], f[3]};
                        else *(u32x2 *)to = u32x2{pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3])};
                    }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                const uint32_t v0 = vw + 32 * j, u0 = uw + UR * p;
                if constexpr (kFactor) {  // u: channels, v: points; eight channels a lane
                    for (int i = 0; i < 32 * UR / 8 / 64; ++i) {
                        const int s = i * 64 + lane, row = s / (UR / 8), c8 = 8 * (s % (UR / 8));
                        const uint32_t pt = v0 + row, c = u0 + c8;
                        if (pt >= V || c >= U) continue;
                        const f32x4 x = *(const f32x4 *)(st + row * PITCH + c8 * 4), y = *(const f32x4 *)(st + row * PITCH + c8 * 4 + 16);
                        const u32x2 k = *(const u32x2 *)(a.kept + (int64_t)pt * a.Cp + c);
                        const float ks = a.kept_scale[pt];
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = (e < 4 ? x[e] : y[e - 4]) * act_slope<ACT>((float)(int8_t)(k[e / 4] >> (8 * (e % 4))) * ks);
                        const u32x4 w = {pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7])};
                        store_run<T, false>((T *)a.out, a.pl, (int64_t)a.X, pt, c, U, w);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32 * PIECES / 64; ++i) {
                        const int s = i * 64 + lane, row = s / PIECES, piece = s % PIECES;
                        const u32x4 w = *(const u32x4 *)(st + row * PITCH + 16 * piece);
                        if (v0 + row >= V) continue;
                        const uint32_t u = u0 + piece * (16 / ES);
                        if constexpr (kF32) store_run<float, false>(a.ws + (int64_t)z * V * U, a.pl, (int64_t)U, v0 + row, u, U, w);
                        else if constexpr (MODE == kInField) {
                            Planes out = a.pl;
                            out.J = V;
                            store_run<T, true>((T *)a.out, out, 0, v0 + row, u, U, w);
                        } else store_run<T, false>((T *)a.out, a.pl, (int64_t)U, v0 + row, u, U, w);
                    }
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
    };
    if constexpr (kFactor) each(std::true_type());
    else if (kWeight && a.splits > 1) each(std::true_type());
    else each(std::false_type());
}

// out = the sum over the splits of their partial sums, four neighbouring values a thread: 16 fours x 16 runs of splits a
// workgroup, joined in LDS in a fixed order.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(const float *ws, int64_t n, int splits, T *out)
{
    __shared__ double part[16][16][4];
    const int t = threadIdx.x, x = t & 15, y = t >> 4;
    const int64_t i = ((int64_t)blockIdx.x * 16 + x) * 4;
    double s[4] = {0, 0, 0, 0};
    const int each = (splits + 15) / 16, z1 = min(splits, (y + 1) * each);
    for (int z = y * each; z < z1; ++z)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < n) s[e] += ws[(int64_t)z * n + i + e];
#pragma unroll
    for (int e = 0; e < 4; ++e) part[y][x][e] = s[e];
    __syncthreads();
    if (y < 4 && i + y < n) {
        double v = 0;
        for (int k = 0; k < 16; ++k) v += part[k][x][y];
        store_elem(out, i + y, (float)v);
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
    a.pl.by_m = fast_div((uint32_t)l.M); a.pl.M = l.M; a.pl.J = l.Co; a.ld = l.Co;
    a.X = (uint32_t)l.C; a.Cp = (int32_t)l.Cp;
    a.splits = 1; a.steps = 0;
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

template <bool F16, int MODE, int ACT>
hipError_t input_tiles(const BwdArgs &a, hipStream_t s)
{
    if (a.X > 128 && ceil_div64(a.A, 256) * ceil_div64(a.X, 256) >= 256) return launch_mode<BLarge, F16, MODE, ACT, false>(a, s);
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
    return l.M > 1 ? input_act<F16, kInField>(l, a, s) : input_act<F16, kInRows>(l, a, s);
}

template <bool F16, int MODE>
hipError_t weight_tiles(const LinearBwdLaunch &l, const BwdArgs &a, hipStream_t s)
{
    if (weight_large(l.Co, l.C))
        return l.db ? launch_mode<BLarge, F16, MODE, DISCO_ACT_NONE, true>(a, s) : launch_mode<BLarge, F16, MODE, DISCO_ACT_NONE, false>(a, s);
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
    const int64_t n = l.Co * l.C;
    join_kernel<T><<<dim3((uint32_t)ceil_div64(n, 64)), dim3(256), 0, s>>>(a.ws, n, p.splits, (T *)l.out);
    if (l.db) join_kernel<T><<<dim3((uint32_t)ceil_div64(l.Co, 64)), dim3(256), 0, s>>>(a.ws_db, l.Co, p.splits, (T *)l.db);
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
