// kernels_linear.hip — the channel product in 8-bit integers:
//
//   y[p][o] = scale[p] wscale[o] sum_c q[p][c] w[o][c] + bias[o]
//
// The sum is exact (32-bit integers, at most 131056 channels); it is converted to fp32, multiplied by the two scales in
// turn, and rounded once more after the bias.
//
// Both operands lie with their channels together, so a tile of rows is 64-byte pieces for the matrix cores' 8-bit
// instruction (v_mfma_i32_32x32x32_i8), brought by direct loads to LDS.  Rows and fields differ in which operand the
// instruction takes first: a lane holds four neighbouring values of its first operand's axis, which is the one that lies
// together in the output, the output channels (rows) or the points (fields).  With few channels a wave's products and its
// writes, from one set of accumulators, take turns (259200 rows, 512 to 2048 bf16: 376 us, 3.2 TB/s and the matrix cores 38 %
// busy; 2x256x721x1440 from 256: 380); many are bound by the matrix cores (8192^3: 558 us, 2.0 Pop/s), few points by the
// weights' bytes (16 rows, 8192 to 8192: 17.4 us, 3.9 TB/s) or the launch.
#include "kernels.hpp"
#include "linear.hpp"
#include "linear_device.hpp"

namespace disco {

namespace {

template <int BU_, int BV_, int WU_, int WV_, int RING_, int K_>
struct LTile {
    static constexpr int BU = BU_, BV = BV_, WU = WU_, WV = WV_, RING = RING_;
    static constexpr int K = K_;                                 // channels of a step
    static constexpr int kThreads = 64 * WU * WV;
    static constexpr int FU = BU / WU / 32, FV = BV / WV / 32;   // 32 x 32 accumulators of a wave
    static constexpr int kU = BU * K, kV = BV * K, kStage = kU + kV;
    static constexpr int LOADS = (BU + BV) * (K / 16) / kThreads; // direct loads of a thread and step
};
typedef LTile<256, 256, 2, 4, 4, 64> LLarge;
typedef LTile<256, 128, 2, 2, 3, 64> LMid;
typedef LTile<128, 128, 2, 2, 4, 64> LSmall;

struct LinArgs {
    const int8_t *uq, *vq;         // rows of Cp bytes
    const float *us, *vs;          // their scales
    const float *bias;             // or null
    void *y;
    Planes pl;                     // the output's points (fields), or its rows
    uint32_t U, V;
    int32_t Cp, nu, nv;            // tiles
    int32_t total;
};

// Rows row0 .. of `rows` of an operand, channels k .. k + 63, to LDS (lin_piece says where).
template <int ROWS, int THREADS, int K>
__device__ __forceinline__ void lin_load(const int8_t *base, uint32_t row0, uint32_t rows, int Cp, int k, unsigned char *dst, int tid, int wave)
{
    // the descriptor starts at the tile's first row, so that offsets stay small however long the tensor is
    const uint32_t left = rows - row0 < (uint32_t)ROWS ? rows - row0 : (uint32_t)ROWS;
    const __amdgpu_buffer_rsrc_t r = lin_rsrc(base + (int64_t)row0 * Cp, left * (uint32_t)Cp);
#pragma unroll
    for (int i = 0; i < ROWS * (K / 16) / THREADS; ++i) {
        const int s = i * THREADS + tid, row = s / (K / 16), piece = lin_piece<K>(s), kk = k + 16 * piece;
        const uint32_t off = (uint32_t)row < left && kk < Cp ? (uint32_t)(row * Cp + kk) : kLinOob;
        lin_dma16(r, off, dst + 16 * (i * THREADS + wave * 64));
    }
}

template <int K>
__device__ __forceinline__ i32x4 lin_frag(const unsigned char *op, int row, int ks, int h)
{
    return *reinterpret_cast<const i32x4 *>(op + lin_at<K>(row, 2 * ks + h));
}

template <typename L, typename T, bool FIELD>
__global__ __launch_bounds__(L::kThreads, 2) void linear_i8_kernel(LinArgs a)
{
    constexpr int FU = L::FU, FV = L::FV, ES = (int)sizeof(T);
    constexpr int UR = FU * 32 * ES > 256 ? 256 / ES : FU * 32;      // u of a staged piece
    constexpr int FP = UR / 32, PITCH = UR * ES + 16, PIECES = UR * ES / 16, kPiece = 32 * PITCH;
    constexpr int kOut = kPiece * L::WU * L::WV, kIn = L::RING * L::kStage;
    __shared__ __attribute__((aligned(16))) unsigned char smem[kOut > kIn ? kOut : kIn];
    __shared__ __attribute__((aligned(16))) float factor[L::BU], addend[L::BU];   // of the tile's u
    int tu, tv;
    if (FIELD) lin_tile(blockIdx.x, a.total, a.nv, &tv, &tu);   // the output channels' tiles of the same points
    else lin_tile(blockIdx.x, a.total, a.nu, &tu, &tv);         // follow each other
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wu = wave % L::WU, wv = wave / L::WU;
    const uint32_t u0 = (uint32_t)tu * L::BU, v0 = (uint32_t)tv * L::BV;
    i32x16 d[FU][FV];
#pragma unroll
    for (int i = 0; i < FU; ++i)
#pragma unroll
        for (int j = 0; j < FV; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) d[i][j][e] = 0;

    const int nk = (a.Cp + L::K - 1) / L::K;
    auto issue = [&](int t) {
        unsigned char *dst = smem + (t % L::RING) * L::kStage;
        lin_load<L::BU, L::kThreads, L::K>(a.uq, u0, a.U, a.Cp, t * L::K, dst, tid, wave);
        lin_load<L::BV, L::kThreads, L::K>(a.vq, v0, a.V, a.Cp, t * L::K, dst + L::kU, tid, wave);
    };
    // asked for first and put down after the sums, so that no step waits for them
    static_assert(L::BU <= L::kThreads, "one u a thread");
    const uint32_t my_u = u0 + tid < a.U ? u0 + tid : a.U - 1;
    const float my_factor = a.us[my_u], my_addend = !FIELD && a.bias ? a.bias[my_u] : 0.0f;
    float vs[FV], vb[FV];
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int j = 0; j < FV; ++j) {
        const uint32_t vw = v0 + L::BV / L::WV * wv + 32 * j + r, v = vw < a.V ? vw : a.V - 1;
        vs[j] = a.vs[v];
        vb[j] = FIELD && a.bias ? a.bias[v] : 0.0f;
    }
#pragma unroll
    for (int t = 0; t < L::RING - 1; ++t)
        if (t < nk) issue(t);
    for (int t = 0; t < nk; ++t) {
        // this thread's loads of step t have landed; those of the steps after it may be in flight
        static_assert(L::RING >= 2 && L::RING <= 4, "up to two steps in flight");
        if (L::RING == 4 && t + 2 < nk) wait_vm<2 * L::LOADS>();
        else if (L::RING > 2 && t + 1 < nk) wait_vm<L::LOADS>();
        else wait_vm<0>();
        bare_barrier();  // everyone's have; and every wave is done with step t - 1, whose place is filled next
        if (t + L::RING - 1 < nk) issue(t + L::RING - 1);
        const unsigned char *cur = smem + (t % L::RING) * L::kStage;
#pragma unroll
        for (int ks = 0; ks < L::K / 32; ++ks) {
            i32x4 fu[FU], fv[FV];
#pragma unroll
            for (int i = 0; i < FU; ++i) fu[i] = lin_frag<L::K>(cur, L::BU / L::WU * wu + 32 * i + r, ks, h);
#pragma unroll
            for (int j = 0; j < FV; ++j) fv[j] = lin_frag<L::K>(cur + L::kU, L::BV / L::WV * wv + 32 * j + r, ks, h);
#pragma unroll
            for (int i = 0; i < FU; ++i)
#pragma unroll
                for (int j = 0; j < FV; ++j) d[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fu[i], fv[j], d[i][j], 0, 0, 0);
        }
    }

    // A lane holds column v = r and rows u = 8 (e / 4) + 4 h + e % 4 of each accumulator: four neighbouring u at a time.
    // Each wave turns 32 v x UR u at a time in LDS of its own, and writes them as runs of 16 bytes along u.
    if (tid < L::BU) {
        factor[tid] = my_factor;
        addend[tid] = my_addend;
    }
    __syncthreads();
    unsigned char *st = smem + wave * kPiece;
    const int uw = L::BU / L::WU * wu;
    const uint32_t vw = v0 + L::BV / L::WV * wv;
#pragma unroll
    for (int p = 0; p < FU / FP; ++p) {
        const RunOut<T, FIELD> out((T *)a.y, a.pl, u0 + uw + UR * p + lane % PIECES * (16 / ES), a.U);
#pragma unroll
        for (int j = 0; j < FV; ++j) {
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int ur = 32 * i + 8 * g + 4 * h;   // within the piece
                    const f32x4 us = *(const f32x4 *)&factor[uw + UR * p + ur], ub = *(const f32x4 *)&addend[uw + UR * p + ur];
                    f32x4 f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float acc = (float)d[FP * p + i][j][4 * g + e];
                        // the point's scale, then the output channel's
                        f[e] = FIELD ? acc * us[e] * vs[j] + vb[j] : acc * vs[j] * us[e] + ub[e];
                    }
                    put4<T>(st + r * PITCH + ur * ES, f);
                }
            // the piece is this wave's own: its LDS operations are done in order
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int i = 0; i < 32 * PIECES / 64; ++i) {
                const int row = i * (64 / PIECES) + lane / PIECES;
                const u32x4 w = *(const u32x4 *)(st + row * PITCH + 16 * (lane % PIECES));
                if (vw + 32 * j + row < a.V) out.put(vw + 32 * j + row, w);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    }
}

// ---------------------------------------------------------------- many points, up to 512 channels

// The weights stay in the matrix cores' registers: a wave holds 64 output channels with all their input channels, a workgroup
// of four 256 of them, and walks a stream of points, PT at a time, which pass through a ring of tiles in LDS (LStay).
struct StayArgs {
    LinArgs l;
    int32_t nt;                      // stores past the caches
    int32_t nb, streams, tiles;      // blocks of output channels, streams, tiles of points
};

template <int KB, typename T, bool FIELD>
__global__ __launch_bounds__(256, 2) void linear_i8_stay_kernel(StayArgs a)
{
    typedef LStay<KB> L;
    constexpr int FX = L::PT / 32, NK = KB / 32, ES = (int)sizeof(T), RING = L::RING;
    constexpr int FU = FIELD ? FX : 2, FV = FIELD ? 2 : FX;                     // frags along u and v
    constexpr int NS = FU * FV * (ES == 2 ? 2 : 4);                             // stores of a wave and tile
    __shared__ __attribute__((aligned(16))) unsigned char ring[RING * L::kStage];
    __shared__ __attribute__((aligned(16))) float factor[kStayChannels], addend[kStayChannels];
    const int64_t me = xcd_tile(blockIdx.x, gridDim.x);   // the blocks of one stream on one XCD
    const int cb = (int)(me % a.nb), stream = (int)(me / a.nb);
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int8_t *wq = FIELD ? a.l.vq : a.l.uq, *xq = FIELD ? a.l.uq : a.l.vq;
    const float *wsc = FIELD ? a.l.vs : a.l.us, *xsc = FIELD ? a.l.us : a.l.vs;
    const uint32_t Co = FIELD ? a.l.V : a.l.U, P = FIELD ? a.l.U : a.l.V;
    const int Cp = a.l.Cp;
    const uint32_t c0 = (uint32_t)cb * kStayChannels + 64 * wave;
    // The streams take the tiles in turn, so that all of them write one region at a time (each a run of its own: addresses a
    // large stride apart meet the same memory channels, 259200 rows 512 to 2048 374 against 364 us, 2076480 rows of 256 349
    // against 298).
    const int n_tiles = (a.tiles - stream + a.streams - 1) / a.streams;

    i32x4 w[2][NK];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const uint32_t c = c0 + 32 * i + r;
            const int kk = 32 * k + 16 * h;
            w[i][k] = c < Co && kk < Cp ? *(const i32x4 *)(wq + (int64_t)c * Cp + kk) : i32x4{0, 0, 0, 0};
        }
    float cs[2], cbias[2];   // fields: of this lane's channels
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t c = c0 + 32 * i + r, cc = c < Co ? c : Co - 1;
        cs[i] = wsc[cc];
        cbias[i] = a.l.bias ? a.l.bias[cc] : 0.0f;
        if (!FIELD && h == 0) {  // rows: four neighbouring channels at a time
            factor[64 * wave + 32 * i + r] = cs[i];
            addend[64 * wave + 32 * i + r] = cbias[i];
        }
    }
    wait_vm<0>();   // the weights are there: no wait for them is left to the loop
    auto issue = [&](int t) {
        unsigned char *dst = ring + t % RING * L::kStage;
        const uint32_t p0 = (uint32_t)(stream + t * a.streams) * L::PT;
        const uint32_t left = P - p0 < (uint32_t)L::PT ? P - p0 : (uint32_t)L::PT;
        const rsrc4_t rx = lin_rsrc4(xq + (int64_t)p0 * Cp, left * (uint32_t)Cp), rs = lin_rsrc4(xsc + p0, left * 4);
        const uint32_t at = lds_offset(dst);
#pragma unroll
        for (int i = 0; i < L::LOADS - 1; ++i) {
            const int s = i * 256 + tid, row = s / (KB / 16), kk = 16 * lin_piece<KB>(s);
            lin_dma16_free(rx, (uint32_t)row < left && kk < Cp ? (uint32_t)(row * Cp + kk) : kLinOob, at + 16 * (i * 256 + wave * 64));
        }
        lin_dma4_free(rs, lane * 4, at + L::kTile + 256 * wave);   // zeros past the end
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i)
        if (i < n_tiles) issue(i);
    int clean = 0;   // how many of the last tiles stored NS times for certain
    for (int t = 0; t < n_tiles; ++t) {
        // This wave's loads of tile t have landed.  What it issued after them may be in flight: the loads of the RING - 2
        // tiles that follow, and the stores of the RING - 1 tiles before this one.
        if (t + RING - 2 >= n_tiles) wait_vm<0>();
        else if (clean == 0) wait_vm<(RING - 2) * L::LOADS>();
        else if (clean == 1) wait_vm<(RING - 2) * L::LOADS + NS>();
        else if (clean == 2 || RING == 3) wait_vm<(RING - 2) * L::LOADS + 2 * NS>();
        else wait_vm<(RING - 2) * L::LOADS + (RING - 1) * NS>();
        bare_barrier();   // everyone's have; and every wave is done with tile t - 1, whose place is filled next
        if (t + RING - 1 < n_tiles) issue(t + RING - 1);
        if (c0 >= Co) continue;
        const unsigned char *cur = ring + t % RING * L::kStage;
        i32x16 d[FU][FV];
        const i32x16 zero = {};
        // four of the points' operands at a time, the next four asked for before their products: alone, the compiler asks for
        // each right before it is used and the products wait for LDS
        constexpr int GK = 4 / FX < NK ? 4 / FX : NK, NG = NK / GK;
        i32x4 x[2][GK][FX];
        auto ask = [&](int g) {
#pragma unroll
            for (int q = 0; q < GK; ++q)
#pragma unroll
                for (int j = 0; j < FX; ++j) x[g & 1][q][j] = lin_frag<KB>(cur, 32 * j + r, g * GK + q, h);
        };
        ask(0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g + 1 < NG) ask(g + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < GK; ++q)
#pragma unroll
                for (int j = 0; j < FX; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = g * GK + q;
                        if constexpr (FIELD) d[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x[g & 1][q][j], w[i][k], k ? d[j][i] : zero, 0, 0, 0);
                        else d[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i][k], x[g & 1][q][j], k ? d[i][j] : zero, 0, 0, 0);
                    }
            __builtin_amdgcn_sched_barrier(0);
        }
        const float *ps = (const float *)(cur + L::kTile + 256 * wave);   // the points' scales
        const uint32_t p0 = (uint32_t)(stream + t * a.streams) * L::PT;
        const uint32_t u0 = FIELD ? p0 : c0, v0 = FIELD ? c0 : p0;
        // every lane's runs are whole and every row is there
        const bool full = p0 + L::PT <= P && c0 + 64 <= Co &&
                          (!FIELD || p0 - a.l.pl.by_m.div(p0) * (uint32_t)a.l.pl.M + L::PT <= (uint32_t)a.l.pl.M);
        const int64_t stride = a.l.pl.template stride<FIELD>();
        T *y = (T *)a.l.y + a.l.pl.template run<FIELD>(u0) + (int64_t)(v0 + frag_v<T, FU>(lane)) * stride + frag_u<T, FU>(lane);
#pragma unroll
        for (int j = 0; j < FV; ++j) {
            const float vs = FIELD ? cs[j] : ps[32 * j + r];
            f32x4 f[FU][4];
#pragma unroll
            for (int i = 0; i < FU; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int ur = 32 * i + 8 * g + 4 * h;
                    if constexpr (FIELD) {
                        const f32x4 us = *(const f32x4 *)&ps[ur];
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[i][g][e] = (float)d[i][j][4 * g + e] * us[e] * vs + cbias[j];
                    } else {
                        const f32x4 us = *(const f32x4 *)&factor[64 * wave + ur], ub = *(const f32x4 *)&addend[64 * wave + ur];
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[i][g][e] = (float)d[i][j][4 * g + e] * vs * us[e] + ub[e];
                    }
                }
            if (full) {
                if (a.nt) store_frag<T, FU, true>(y + (int64_t)(32 * j) * stride, stride, f);
                else store_frag<T, FU, false>(y + (int64_t)(32 * j) * stride, stride, f);
            } else {
#pragma unroll
                for (int i = 0; i < FU; ++i)
                    store_frag_part<T, FIELD>((T *)a.l.y, a.l.pl, lane, u0 + 32 * i, a.l.U, v0 + 32 * j, a.l.V, f[i]);
            }
        }
        clean = full ? clean + 1 : 0;
    }
}

// ---------------------------------------------------------------- few points

// Up to 16 MT points against all weights, each weight read once: a workgroup takes 16 output channels, its eight waves
// a share of the input channels each, straight from memory into the matrix cores' registers; the shares are joined in LDS
// (whole numbers: the order does not matter).
constexpr int kFewSteps = 4;   // steps of 64 channels asked for in one go

template <typename T, int MT, bool FIELD>
__global__ __launch_bounds__(64 * kFewWaves) void linear_i8_few_kernel(LinArgs a, int lg_run)
{
    __shared__ __attribute__((aligned(16))) int part[kFewWaves][MT][64][4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int8_t *wq = FIELD ? a.vq : a.uq, *xq = FIELD ? a.uq : a.vq;
    const float *wsc = FIELD ? a.vs : a.us, *xs = FIELD ? a.us : a.vs;
    const uint32_t Co = FIELD ? a.V : a.U, Pn = FIELD ? a.U : a.V;
    const uint32_t o0 = blockIdx.x * 16;
    const uint32_t o = o0 + (lane & 15), oc = o < Co ? o : Co - 1;
    const int kq = 16 * (lane >> 4);
    i32x4 d[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) d[m] = i32x4{0, 0, 0, 0};
    const i32x4 zero = {0, 0, 0, 0};
    const int8_t *wr = wq + (int64_t)oc * a.Cp;
    // a wave's steps lie together in runs of 2^lg_run channels
    const int run = 1 << lg_run;
    for (int k0 = 0; k0 < a.Cp; k0 += 64 * kFewWaves * kFewSteps) {
        i32x4 fw[kFewSteps], fx[kFewSteps][MT];
#pragma unroll
        for (int s = 0; s < kFewSteps; ++s) {
            const int kk = k0 + ((64 * s >> lg_run) * kFewWaves + wave) * run + (64 * s & (run - 1)) + kq;
            const bool in = kk < a.Cp;
            fw[s] = in ? *(const i32x4 *)(wr + kk) : zero;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t p = 16 * m + (lane & 15);
                fx[s][m] = in && p < Pn ? *(const i32x4 *)(xq + (int64_t)p * a.Cp + kk) : zero;
            }
        }
#pragma unroll
        for (int s = 0; s < kFewSteps; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m) d[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[s], fx[s][m], d[m], 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) *(i32x4 *)part[wave][m][lane] = d[m];
    __syncthreads();
    // a lane holds column p = lane % 16 and rows o = 4 (lane / 16) + e
    for (int i = tid; i < MT * 64; i += 64 * kFewWaves) {
        const int m = i >> 6, l = i & 63;
        i32x4 s = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) s += *(const i32x4 *)part[w][m][l];
        const uint32_t p = 16 * m + (l & 15);
        if (p >= Pn) continue;
        const float ps = xs[p];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t oo = o0 + 4 * (l >> 4) + e;
            if (oo < Co) {
                const float v = (float)s[e] * ps * wsc[oo] + (a.bias ? a.bias[oo] : 0.0f);
                store_elem((T *)a.y, FIELD ? a.pl.run<true>(p) + oo * a.pl.M : (int64_t)p * a.pl.ld + oo, v);
            }
        }
    }
}

template <typename L, typename T, bool FIELD>
hipError_t launch_tiles(LinArgs a, hipStream_t s)
{
    a.nu = (int32_t)(((int64_t)a.U + L::BU - 1) / L::BU);
    a.nv = (int32_t)(((int64_t)a.V + L::BV - 1) / L::BV);
    a.total = a.nu * a.nv;
    linear_i8_kernel<L, T, FIELD><<<dim3((uint32_t)a.total), dim3(L::kThreads), 0, s>>>(a);
    return hipGetLastError();
}

// Whether runs of the output are whole sectors, and many.
template <typename T, bool FIELD>
bool stays_whole(const LinArgs &l)
{
    return stream_stores(!FIELD, (int64_t)l.U * l.V * (int64_t)sizeof(T), (FIELD ? l.pl.M : l.pl.ld) * (int64_t)sizeof(T), l.y, nullptr);
}

template <int KB, typename T, bool FIELD>
hipError_t launch_stay(const LinArgs &l, hipStream_t s)
{
    const int64_t P = FIELD ? l.U : l.V, Co = FIELD ? l.V : l.U;
    StayArgs a;
    a.l = l;
    // 16 bits: a store writes whole lines (259200 rows 512 to 2048 404 -> 364 us past the caches; fp32, half a line a store,
    // 512 to 512, 151 -> 177)
    a.nt = sizeof(T) == 2 && stays_whole<T, FIELD>(l);
    a.nb = (int32_t)ceil_div64(Co, kStayChannels);
    a.tiles = (int32_t)ceil_div64(P, LStay<KB>::PT);
    const int64_t streams = a.nb < 512 ? 512 / a.nb : 1;   // two workgroups a CU
    a.streams = (int32_t)(streams < a.tiles ? streams : a.tiles);
    linear_i8_stay_kernel<KB, T, FIELD><<<dim3((uint32_t)(a.nb * a.streams)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

// Which kernel: 128 points at most, each weight is read once (few).  Else, up to 512 channels and points for every stream,
// the weights stay in registers (259200 rows, 512 to 2048, bf16: 364 us against 495 in tiles of 256 x 128); fields where the
// output is stored past the caches (721x1440, 80 to 512: 288 against 296 us; 2x720x1440, 256 to 256: 343 against 389), or from
// 257 channels on (360x720, 512 to 2048: 417 against 531): else the tile's runs of points are the longer ones.  Else tiles:
// 256 x 256 where there is one for every CU and the channels are many (8192^3: 558 us against 762), 256 x 128 where there is
// one for every CU (4x181x360 fields, 32 to 64: 14.6 against 16.9), 128 x 128 (1000 rows, 1024 to 1024: 8.6 against 13.1).
template <typename T, bool FIELD>
hipError_t launch_typed(const LinearLaunch &l, const LinArgs &a, hipStream_t s)
{
    if (l.P <= kFewPoints) {
        const dim3 grid((uint32_t)ceil_div64(l.Co, 16)), block(64 * kFewWaves);
        const int lg = l.Cp >= 2048 ? 8 : 6;   // 16 rows, 8192 to 8192: 17.8 us in runs of 256 channels, 19.0 in runs of 64
        if (l.P <= 16) linear_i8_few_kernel<T, 1, FIELD><<<grid, block, 0, s>>>(a, lg);
        else if (l.P <= 32) linear_i8_few_kernel<T, 2, FIELD><<<grid, block, 0, s>>>(a, lg);
        else if (l.P <= 64) linear_i8_few_kernel<T, 4, FIELD><<<grid, block, 0, s>>>(a, lg);
        else linear_i8_few_kernel<T, 8, FIELD><<<grid, block, 0, s>>>(a, lg);
        return hipGetLastError();
    }
    if (l.Cp <= 512 && (!FIELD || l.Cp > 256 || (sizeof(T) == 2 && stays_whole<T, FIELD>(a))) && l.P * ceil_div64(l.Co, kStayChannels) >= 512 * 64)
        return l.Cp <= 64 ? launch_stay<64, T, FIELD>(a, s) : l.Cp <= 128 ? launch_stay<128, T, FIELD>(a, s)
             : l.Cp <= 256 ? launch_stay<256, T, FIELD>(a, s) : launch_stay<512, T, FIELD>(a, s);
    if (l.Cp > 512 && ceil_div64(l.P, 256) * ceil_div64(l.Co, 256) >= 256) return launch_tiles<LLarge, T, FIELD>(a, s);
    if (ceil_div64(a.U, 256) * ceil_div64(a.V, 128) >= 256) return launch_tiles<LMid, T, FIELD>(a, s);
    return launch_tiles<LSmall, T, FIELD>(a, s);
}

}  // namespace

hipError_t launch_linear_i8(const LinearLaunch &l, hipStream_t s)
{
    const bool field = l.M > 1;
    LinArgs a;
    a.uq = field ? l.q : l.w; a.us = field ? l.scale : l.wscale;
    a.vq = field ? l.w : l.q; a.vs = field ? l.wscale : l.scale;
    a.bias = (const float *)l.bias; a.y = l.y;
    a.pl.by_m = fast_div((uint32_t)l.M); a.pl.M = l.M; a.pl.J = l.Co; a.pl.ld = l.Co;
    a.U = (uint32_t)(field ? l.P : l.Co); a.V = (uint32_t)(field ? l.Co : l.P);
    a.Cp = (int32_t)l.Cp; a.nu = a.nv = a.total = 0;
    if (field)
        return l.dtype == 0 ? launch_typed<float, true>(l, a, s) : l.dtype == 1 ? launch_typed<bf16_t, true>(l, a, s) : launch_typed<f16_t, true>(l, a, s);
    return l.dtype == 0 ? launch_typed<float, false>(l, a, s) : l.dtype == 1 ? launch_typed<bf16_t, false>(l, a, s) : launch_typed<f16_t, false>(l, a, s);
}

}  // namespace disco
