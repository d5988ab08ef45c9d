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
// together in the output, the output channels (rows) or the points (fields).
#include "kernels.hpp"
#include "linear.hpp"
#include "linear_device.hpp"

namespace disco {

namespace {

constexpr int kLK = 64;   // channels of a step

template <int BU_, int BV_, int WU_, int WV_, int RING_>
struct LTile {
    static constexpr int BU = BU_, BV = BV_, WU = WU_, WV = WV_, RING = RING_;
    static constexpr int kThreads = 64 * WU * WV;
    static constexpr int FU = BU / WU / 32, FV = BV / WV / 32;   // 32 x 32 accumulators of a wave
    static constexpr int kU = BU * kLK, kV = BV * kLK, kStage = kU + kV;
    static constexpr int LOADS = (BU + BV) * 4 / kThreads;       // direct loads of a thread and step
};
typedef LTile<256, 256, 2, 4, 4> LLarge;
typedef LTile<128, 128, 2, 2, 4> LSmall;

struct LinArgs {
    const int8_t *uq, *vq;         // rows of Cp bytes
    const float *us, *vs;          // their scales
    const float *bias;             // or null
    void *y;
    Planes pl;                     // fields: the points' planes
    int64_t ld;                    // rows: the output's row
    uint32_t U, V;
    int32_t Cp, nu, nv;            // tiles
    int32_t u_fast;                // which tiles follow each other
    int32_t total;
};

// Rows row0 .. of `rows` of an operand, channels k .. k + 63, to LDS (lin_piece says where).
template <int ROWS, int THREADS>
__device__ __forceinline__ void lin_load(const int8_t *base, uint32_t row0, uint32_t rows, int Cp, int k, unsigned char *dst, int tid, int wave)
{
    // the descriptor starts at the tile's first row, so that offsets stay small however long the tensor is
    const uint32_t left = rows - row0 < (uint32_t)ROWS ? rows - row0 : (uint32_t)ROWS;
    const __amdgpu_buffer_rsrc_t r = lin_rsrc(base + (int64_t)row0 * Cp, left * (uint32_t)Cp);
#pragma unroll
    for (int i = 0; i < ROWS * 4 / THREADS; ++i) {
        const int s = i * THREADS + tid, row = s >> 2, piece = lin_piece(s), kk = k + 16 * piece;
        const uint32_t off = (uint32_t)row < left && kk < Cp ? (uint32_t)(row * Cp + kk) : kLinOob;
        lin_dma16(r, off, dst + 16 * (i * THREADS + wave * 64));
    }
}

__device__ __forceinline__ i32x4 lin_frag(const unsigned char *op, int row, int ks, int h)
{
    return *reinterpret_cast<const i32x4 *>(op + lin_at(row, 2 * ks + h));
}

template <typename T>
__device__ __forceinline__ u32x2 pack4(float a, float b, float c, float d)
{
    const float f[4] = {a, b, c, d};
    Pack<T, 4> p;
    pack(f, p);
    return {p.w[0], p.w[1]};
}

// The values of one 32 (v) x UR (u) piece of a wave, staged in LDS as rows of u, to memory in 16-byte pieces.
template <typename T, bool PLANES, int UR>
__device__ __forceinline__ void lin_write(const unsigned char *st, int lane, T *y, const Planes &pl, int64_t ld, uint32_t v0, uint32_t V,
                                          uint32_t u0, uint32_t U)
{
    constexpr int PITCH = UR * (int)sizeof(T) + 16, PIECES = UR * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < 32 * PIECES / 64; ++i) {
        const int s = i * 64 + lane, row = s / PIECES, piece = s % PIECES;
        const u32x4 w = *reinterpret_cast<const u32x4 *>(st + row * PITCH + 16 * piece);
        if (v0 + row < V) store_run<T, PLANES>(y, pl, ld, v0 + row, u0 + piece * (16 / (int)sizeof(T)), U, w);
    }
}

template <typename L, typename T, bool FIELD>
__global__ __launch_bounds__(L::kThreads) void linear_i8_kernel(LinArgs a)
{
    constexpr int FU = L::FU, FV = L::FV;
    constexpr int UR = FU * 32 * (int)sizeof(T) > 256 ? 256 / (int)sizeof(T) : FU * 32;  // u of a staged piece
    constexpr int kPiece = 32 * (UR * (int)sizeof(T) + 16);
    constexpr int kOut = kPiece * L::WU * L::WV, kIn = L::RING * L::kStage;
    __shared__ __attribute__((aligned(16))) unsigned char smem[kOut > kIn ? kOut : kIn];
    int tu, tv;
    if (a.u_fast) lin_tile(blockIdx.x, a.total, a.nu, &tu, &tv);
    else lin_tile(blockIdx.x, a.total, a.nv, &tv, &tu);
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

    const int nk = (a.Cp + kLK - 1) / kLK;
    auto issue = [&](int t) {
        unsigned char *dst = smem + (t % L::RING) * L::kStage;
        lin_load<L::BU, L::kThreads>(a.uq, u0, a.U, a.Cp, t * kLK, dst, tid, wave);
        lin_load<L::BV, L::kThreads>(a.vq, v0, a.V, a.Cp, t * kLK, dst + L::kU, tid, wave);
    };
#pragma unroll
    for (int t = 0; t < L::RING - 1; ++t)
        if (t < nk) issue(t);
    const int r = lane & 31, h = lane >> 5;
    for (int t = 0; t < nk; ++t) {
        // this thread's loads of step t have landed; those of the steps after it may be in flight
        static_assert(L::LOADS == 4 && L::RING == 4, "the waits below count steps of four loads");
        if (t + 2 < nk) __builtin_amdgcn_s_waitcnt(0x078);        // vmcnt 8, lgkmcnt 0
        else if (t + 1 < nk) __builtin_amdgcn_s_waitcnt(0x074);   // vmcnt 4
        else __builtin_amdgcn_s_waitcnt(0x070);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();  // everyone's have; and every wave is done with step t - 1, whose place is filled next
        asm volatile("" ::: "memory");
        if (t + L::RING - 1 < nk) issue(t + L::RING - 1);
        const unsigned char *cur = smem + (t % L::RING) * L::kStage;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            i32x4 fu[FU], fv[FV];
#pragma unroll
            for (int i = 0; i < FU; ++i) fu[i] = lin_frag(cur, L::BU / L::WU * wu + 32 * i + r, ks, h);
#pragma unroll
            for (int j = 0; j < FV; ++j) fv[j] = lin_frag(cur + L::kU, L::BV / L::WV * wv + 32 * j + r, ks, h);
#pragma unroll
            for (int i = 0; i < FU; ++i)
#pragma unroll
                for (int j = 0; j < FV; ++j) d[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fu[i], fv[j], d[i][j], 0, 0, 0);
        }
    }

    // A lane holds column v = r and rows u = 8 (e / 4) + 4 h + e % 4 of each accumulator: four neighbouring u at a time.
    __syncthreads();
    unsigned char *st = smem + wave * kPiece;
    constexpr int PITCH = UR * (int)sizeof(T) + 16, FP = UR / 32;
    const uint32_t uw = u0 + L::BU / L::WU * wu, vw = v0 + L::BV / L::WV * wv;
#pragma unroll
    for (int j = 0; j < FV; ++j) {
        const uint32_t v = vw + 32 * j + r;
        const float vs = a.vs[v < a.V ? v : a.V - 1];
        const float vb = FIELD && a.bias ? a.bias[v < a.V ? v : a.V - 1] : 0.0f;
#pragma unroll
        for (int p = 0; p < FU / FP; ++p) {
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int ur = 32 * i + 8 * g + 4 * h;   // within the piece
                    float f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u = uw + UR * p + ur + e, uc = u < a.U ? u : a.U - 1;
                        const float acc = (float)d[FP * p + i][j][4 * g + e];
                        // the point's scale, then the output channel's
                        f[e] = FIELD ? acc * a.us[uc] * vs : acc * vs * a.us[uc];
                        f[e] += FIELD ? vb : a.bias ? a.bias[uc] : 0.0f;
                    }
                    unsigned char *to = st + r * PITCH + ur * (int)sizeof(T);
                    if constexpr (sizeof(T) == 4) *(f32x4 *)to = f32x4{f[0], f[1], f[2], f[3]};
                    else *(u32x2 *)to = pack4<T>(f[0], f[1], f[2], f[3]);
                }
            // the piece is this wave's own: its LDS writes are in order before its reads
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            lin_write<T, FIELD, UR>(st, lane, (T *)a.y, a.pl, a.ld, vw + 32 * j, a.V, uw + UR * p, a.U);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    }
}

// ---------------------------------------------------------------- few points

// Up to 16 MT points against all weights, each weight read once: a workgroup takes 16 output channels, its eight waves
// a share of the input channels each, straight from memory into the matrix cores' registers; the shares are joined in LDS
// (whole numbers: the order does not matter).
constexpr int kFewWaves = 8;

template <typename T, int MT, bool FIELD>
__global__ __launch_bounds__(64 * kFewWaves) void linear_i8_few_kernel(LinArgs a)
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
#pragma unroll 4
    for (int k = 64 * wave; k < a.Cp; k += 64 * kFewWaves) {
        const int kk = k + kq;
        const bool in = kk < a.Cp;
        const i32x4 fw = in ? *(const i32x4 *)(wr + kk) : zero;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t p = 16 * m + (lane & 15);
            const i32x4 fx = in && p < Pn ? *(const i32x4 *)(xq + (int64_t)p * a.Cp + kk) : zero;
            d[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw, fx, d[m], 0, 0, 0);
        }
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
                store_elem((T *)a.y, FIELD ? a.pl.at(oo, p) : (int64_t)p * a.ld + oo, v);
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
    a.u_fast = FIELD ? 0 : 1;   // the output channels' tiles of the same points follow each other
    linear_i8_kernel<L, T, FIELD><<<dim3((uint32_t)a.total), dim3(L::kThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool FIELD>
hipError_t launch_typed(const LinearLaunch &l, const LinArgs &a, hipStream_t s)
{
    if (l.P <= 64) {
        const dim3 grid((uint32_t)ceil_div64(l.Co, 16)), block(64 * kFewWaves);
        if (l.P <= 16) linear_i8_few_kernel<T, 1, FIELD><<<grid, block, 0, s>>>(a);
        else if (l.P <= 32) linear_i8_few_kernel<T, 2, FIELD><<<grid, block, 0, s>>>(a);
        else linear_i8_few_kernel<T, 4, FIELD><<<grid, block, 0, s>>>(a);
        return hipGetLastError();
    }
    if (ceil_div64(l.P, 256) * ceil_div64(l.Co, 256) >= 256 && l.Co > 128) return launch_tiles<LLarge, T, FIELD>(a, s);
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
    a.pl.by_m = fast_div((uint32_t)l.M); a.pl.M = l.M; a.pl.J = l.Co; a.ld = l.Co;
    a.U = (uint32_t)(field ? l.P : l.Co); a.V = (uint32_t)(field ? l.Co : l.P);
    a.Cp = (int32_t)l.Cp; a.nu = a.nv = a.u_fast = a.total = 0;
    if (field)
        return l.dtype == 0 ? launch_typed<float, true>(l, a, s) : l.dtype == 1 ? launch_typed<bf16_t, true>(l, a, s) : launch_typed<f16_t, true>(l, a, s);
    return l.dtype == 0 ? launch_typed<float, false>(l, a, s) : l.dtype == 1 ? launch_typed<bf16_t, false>(l, a, s) : launch_typed<f16_t, false>(l, a, s);
}

}  // namespace disco
