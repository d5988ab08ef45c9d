// kernels_linear_bwd_stay.hip — the gradient of the channel product's input over many rows, for up to 512 output channels:
//
//   gx[p][c] = act'(kept[p][c]) sum_o gy[p][o] (wscale[o] w[o][c])
//
// The weights (rounded once to the data type, as in the tiles of kernels_linear_bwd.hip) are formed once a workgroup and stay in
// the matrix cores' registers: a wave holds 64 input channels (32 beyond 256 output channels), a workgroup of four walks a
// stream of points whose gradients and checkpoints pass through a ring of tiles in LDS by direct loads.  In tiles, a third of
// the vector instructions form the weights again for every 256 points, and with gelu's slope they, not the matrix cores, are
// the bound.  bf16, us against tiles: 259200 rows, 2048 from 512, 935 against 1067 with gelu, 700 against 743 alone; 1000000
// rows with gelu, 512 from 128, 523 against 696, 256 from 64, 230 against 315; 2076480 rows, 256 from 256, 468 against 535.
// With gelu at 2048 from 512 the matrix cores work a quarter of the time (0.58 PFLOP/s) and half of the waves' time is waits.
#include <type_traits>

#include "act_device.hpp"
#include "kernels.hpp"
#include "linear.hpp"
#include "linear_device.hpp"

namespace disco {

namespace {

struct GStayArgs {
    const uint16_t *gy;
    const int8_t *w, *kept;
    const float *wscale, *kept_scale;
    void *gx;
    Planes pl;                   // gx's rows
    uint32_t P, C, Co;
    int32_t Cp, nt, nb, streams, tiles;
};

template <int KB, bool F16, int ACT>
__global__ __launch_bounds__(256, 2) void linear_bwd_stay_kernel(GStayArgs a)
{
    typedef typename std::conditional<F16, f16_t, bf16_t>::type T;
    constexpr bool KEPT = ACT != DISCO_ACT_NONE;
    typedef GStay<KB, KEPT> L;
    constexpr int FW = L::FW, FX = L::PT / 32, NK = KB / 32, RING = L::RING;
    constexpr int LOADS = L::LOADS + L::KLOADS + (KEPT ? 1 : 0), NS = FW * FX * 2;
    __shared__ __attribute__((aligned(16))) unsigned char ring[RING * L::kStage];
    const int64_t me = xcd_tile(blockIdx.x, gridDim.x);   // the blocks of one stream on one XCD
    const int cb = (int)(me % a.nb), stream = (int)(me / a.nb);
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t b0 = (uint32_t)cb * L::CB, c0 = b0 + L::CW * wave;
    // the streams take the tiles in turn
    const int n_tiles = (a.tiles - stream + a.streams - 1) / a.streams;

    bf16x8 w[FW][NK];
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        float sc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t o = 16 * k + 8 * h + e;
            sc[e] = a.wscale[o < a.Co ? o : a.Co - 1];
        }
#pragma unroll
        for (int i = 0; i < FW; ++i) {
            const uint32_t c = c0 + 32 * i + r;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t o = 16 * k + 8 * h + e;
                v[e] = o < a.Co && c < (uint32_t)a.Cp ? (float)a.w[(int64_t)o * a.Cp + c] * sc[e] : 0.0f;
            }
            const u32x4 p = {pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]), pack2<F16>(v[4], v[5]), pack2<F16>(v[6], v[7])};
            w[i][k] = __builtin_bit_cast(bf16x8, p);
        }
        if (k & 1) __builtin_amdgcn_sched_barrier(0);   // (all bytes asked for at once would not fit beside the weights)
    }
    wait_vm<0>();   // the weights are there: no wait for them is left to the loop
    auto issue = [&](int t) {
        unsigned char *dst = ring + t % RING * L::kStage;
        const uint32_t p0 = (uint32_t)(stream + t * a.streams) * L::PT;
        const uint32_t left = a.P - p0 < (uint32_t)L::PT ? a.P - p0 : (uint32_t)L::PT;
        const int row_bytes = (int)a.Co * 2;
        const rsrc4_t rg = lin_rsrc4(a.gy + (int64_t)p0 * a.Co, left * (uint32_t)row_bytes);
        const uint32_t at = lds_offset(dst);
#pragma unroll
        for (int i = 0; i < L::LOADS; ++i) {
            const int s = i * 256 + tid, row = s / (KB / 16), kk = 16 * lin_piece<KB>(s);
            lin_dma16_free(rg, (uint32_t)row < left && kk < row_bytes ? (uint32_t)(row * row_bytes + kk) : kLinOob, at + 16 * (i * 256 + wave * 64));
        }
        if constexpr (KEPT) {
            const rsrc4_t rk = lin_rsrc4(a.kept + (int64_t)p0 * a.Cp, left * (uint32_t)a.Cp);
#pragma unroll
            for (int i = 0; i < L::KLOADS; ++i) {
                const int s = i * 256 + tid, row = s / (L::CB / 16);
                const uint32_t c = b0 + 16 * lin_piece<L::CB>(s);
                lin_dma16_free(rk, (uint32_t)row < left && c < (uint32_t)a.Cp ? row * (uint32_t)a.Cp + c : kLinOob, at + L::kTile + 16 * (i * 256 + wave * 64));
            }
            lin_dma4_free(lin_rsrc4(a.kept_scale + p0, left * 4), lane * 4, at + L::kTile + L::kKept + 256 * wave);   // zeros past the end
        }
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i)
        if (i < n_tiles) issue(i);
    int clean = 0;   // how many of the last tiles stored NS times for certain
    for (int t = 0; t < n_tiles; ++t) {
        // This wave's loads of tile t have landed.  What it issued after them may be in flight: the loads of the RING - 2
        // tiles that follow, and the stores of the RING - 1 tiles before this one.
        if (t + RING - 2 >= n_tiles) wait_vm<0>();
        else if (clean == 0) wait_vm<(RING - 2) * LOADS>();
        else if (clean == 1 || RING == 2) wait_vm<(RING - 2) * LOADS + NS>();
        else wait_vm<(RING - 2) * LOADS + (RING - 1) * NS>();
        bare_barrier();   // everyone's have; and every wave is done with tile t - 1, whose place is filled next
        if (t + RING - 1 < n_tiles) issue(t + RING - 1);
        if (c0 >= a.C) continue;
        const unsigned char *cur = ring + t % RING * L::kStage;
        f32x16 d[FW][FX];
        const f32x16 zero = {};
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int j = 0; j < FX; ++j) {
                const bf16x8 x = *reinterpret_cast<const bf16x8 *>(cur + lin_at<KB>(32 * j + r, 2 * k + h));
#pragma unroll
                for (int i = 0; i < FW; ++i) d[i][j] = bwd_mma<F16>(w[i][k], x, k ? d[i][j] : zero);
            }
        const uint32_t p0 = (uint32_t)(stream + t * a.streams) * L::PT;
        const bool full = p0 + L::PT <= a.P && c0 + L::CW <= a.C;   // every lane's runs are whole and every row is there
        const int64_t stride = a.pl.ld;
        T *y = (T *)a.gx + c0 + (int64_t)(p0 + frag_v<T, FW>(lane)) * stride + frag_u<T, FW>(lane);
        const unsigned char *kt = cur + L::kTile;
        const float *ks = (const float *)(kt + L::kKept + 256 * wave);
#pragma unroll
        for (int j = 0; j < FX; ++j) {
            const float s = KEPT ? ks[32 * j + r] : 0.0f;
            f32x4 f[FW][4];
#pragma unroll
            for (int i = 0; i < FW; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t q = 0;
                    if constexpr (KEPT) {
                        const int col = L::CW * wave + 32 * i + 8 * g + 4 * h;
                        q = *(const uint32_t *)(kt + lin_at<L::CB>(32 * j + r, col >> 4) + (col & 15));
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[i][g][e] = d[i][j][4 * g + e];
                        if constexpr (KEPT) f[i][g][e] *= act_slope<ACT>((float)(int8_t)(q >> (8 * e)) * s);
                    }
                }
            if (full) {
                if (a.nt) store_frag<T, FW, true>(y + (int64_t)(32 * j) * stride, stride, f);
                else store_frag<T, FW, false>(y + (int64_t)(32 * j) * stride, stride, f);
            } else {
#pragma unroll
                for (int i = 0; i < FW; ++i) store_frag_part<T, false>((T *)a.gx, a.pl, lane, c0 + 32 * i, a.C, p0 + 32 * j, a.P, f[i]);
            }
        }
        clean = full ? clean + 1 : 0;
    }
}

template <int KB, bool F16, int ACT>
hipError_t launch_act(GStayArgs a, hipStream_t s)
{
    typedef GStay<KB, ACT != DISCO_ACT_NONE> L;
    a.nb = (int32_t)ceil_div64(a.C, L::CB);
    a.tiles = (int32_t)ceil_div64(a.P, L::PT);
    if (L::FW == 1) a.nt = 0;   // half lines: past the caches they are written as two (1.50 GB written for 1.06)
    const int64_t streams = a.nb < 512 ? 512 / a.nb : 1;   // two workgroups a CU
    a.streams = (int32_t)(streams < a.tiles ? streams : a.tiles);
    linear_bwd_stay_kernel<KB, F16, ACT><<<dim3((uint32_t)(a.nb * a.streams)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <int KB, bool F16>
hipError_t launch_kb(int act, const GStayArgs &a, hipStream_t s)
{
    return act == DISCO_ACT_GELU ? launch_act<KB, F16, DISCO_ACT_GELU>(a, s)
         : act == DISCO_ACT_SILU ? launch_act<KB, F16, DISCO_ACT_SILU>(a, s)
                                 : launch_act<KB, F16, DISCO_ACT_NONE>(a, s);
}

template <bool F16>
hipError_t launch_typed(int act, const GStayArgs &a, hipStream_t s)
{
    return a.Co <= 64 ? launch_kb<128, F16>(act, a, s) : a.Co <= 128 ? launch_kb<256, F16>(act, a, s)
         : a.Co <= 256 ? launch_kb<512, F16>(act, a, s) : launch_kb<1024, F16>(act, a, s);
}

}  // namespace

// Rows of whole 16-byte pieces, and a tile for every stream.  A tile's checkpoints (64 points) lie behind one 32-bit size and
// offset: longer rows than 2^24 go to the tiles, whose offsets have 64 bits.
bool bwd_stays(const LinearBwdLaunch &l)
{
    return l.M == 1 && l.Co <= 512 && l.Co % 8 == 0 && ((uintptr_t)l.gy & 15) == 0 && l.P * ceil_div64(l.C, 256) >= 512 * 64 &&
           (!l.kept || l.Cp <= 1 << 24);
}

hipError_t launch_linear_bwd_stay(const LinearBwdLaunch &l, bool nt, hipStream_t s)
{
    GStayArgs a;
    a.gy = (const uint16_t *)l.gy; a.w = l.q; a.wscale = l.scale; a.kept = l.kept; a.kept_scale = l.kept_scale; a.gx = l.out;
    a.pl.M = 1; a.pl.J = 1; a.pl.ld = l.C;
    a.P = (uint32_t)l.P; a.C = (uint32_t)l.C; a.Co = (uint32_t)l.Co; a.Cp = (int32_t)l.Cp;
    a.nt = nt; a.nb = a.streams = a.tiles = 0;
    return l.dtype == 2 ? launch_typed<true>(l.act, a, s) : launch_typed<false>(l.act, a, s);
}

}  // namespace disco
