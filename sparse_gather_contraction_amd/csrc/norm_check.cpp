// norm_check.cpp — replays the index arithmetic of the norm kernels on the CPU.
//
//   norm_check            (built by the tests with g++ and the address and undefined-behaviour sanitizers)
//
// For many (N, D, M) and element sizes, walks every workgroup, thread, vector and element of the forward, the
// backward and the 8-bit reader as the kernels do, and checks that every access lies inside the tensor, that
// every element is held exactly once beside its duplicates, that the LDS indexes lie inside the LDS a
// launch asks for, and that this is at most 64 KiB.  Prints the number of geometries checked.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "norm_plan.hpp"

using namespace disco;

static void fail(const char *what, int64_t N, int64_t D, int64_t M, int esz)
{
    printf("FAILED: %s at N=%lld D=%lld M=%lld esz=%d\n", what, (long long)N, (long long)D, (long long)M, esz);
    exit(1);
}

#define REQUIRE(x) do { if (!(x)) fail(#x, N, D, M, esz); } while (0)

static void check_norm(int64_t N, int64_t D, int64_t M, int esz, bool bwd)
{
    const NormGeom g = norm_geom(N, D, M, esz, bwd);
    const int lanes = 1 << g.lg;
    REQUIRE(g.threads >= 64 && g.threads <= kNormMaxThreads && g.threads % 64 == 0 && g.threads >= lanes);
    REQUIRE(g.groups == g.threads >> g.lg && g.tiles >= 1);
    std::vector<int> held((size_t)(N * D * M), 0);
    const int64_t ngs[3] = {1, ceil_div64(D, 32), ceil_div64(D, 96)};
    for (int64_t ng : ngs) {
        const size_t lds = bwd ? norm_bwd_lds(g, D) : norm_lds(g, (int)ng);
        REQUIRE(lds <= 64 * 1024);
        const size_t P = (size_t)lanes * g.vec;
        if (g.loop) {
            REQUIRE((g.groups & (g.groups - 1)) == 0 && lanes <= 64);
            REQUIRE(lds >= (bwd ? 2 : 1) * (size_t)g.groups * P * 4 + (bwd ? 0 : P * 4));
        } else if (g.rows) {
            if (bwd && g.groups > 1) REQUIRE(lds >= (size_t)g.groups * D * 8);
            if (bwd && g.groups == 1 && g.per == 4 && g.vec == 4) REQUIRE(lds >= (size_t)kBwdLdsWeights * g.threads * 16);
        } else {
            const int lg6 = g.lg < 6 ? 6 : g.lg, parts = g.threads >> lg6;
            REQUIRE(parts * (1 << lg6) == g.threads);
            REQUIRE(lds >= (bwd ? (2 * (size_t)parts + 2) : (size_t)parts + 1 + ng) * P * 4);
            // dw: leader lanes write [lane >> 6][g * per + j]
            if (bwd) REQUIRE(lds >= ((size_t)((lanes - 1) >> 6) * g.groups * g.per + (size_t)g.groups * g.per) * 8);
            REQUIRE((int64_t)g.groups * g.per >= D && 32 % g.per == 0);
        }
    }
    for (int64_t tile = 0; tile < g.tiles; ++tile) {
        for (int t = 0; t < g.threads; ++t) {
            const int lane = t & (lanes - 1), grp = t >> g.lg;
            if (g.rows) {
                const int64_t want = tile * g.groups + grp, row = want < N ? want : N - 1;
                for (int k = 0; k < g.per; ++k) {
                    const RowPos p = row_pos(k * lanes + lane, g.vec, (int)D);
                    REQUIRE(p.dup >= 0 && p.c >= 0 && p.c + g.vec <= D);
                    for (int e = p.dup; e < g.vec; ++e)
                        if (want < N) ++held[(size_t)(row * D + p.c + e)];
                }
            } else {
                const ColPos p = col_pos(tile, lane, g.vec, g.lg, g.tiles_n, N, M);
                REQUIRE(p.n >= 0 && p.n < N && p.m >= 0 && p.m + g.vec <= M && p.dup >= 0);
                auto hold = [&](int64_t c) {
                    for (int e = p.dup; e < g.vec; ++e) ++held[(size_t)((p.n * D + c) * M + p.m + e)];
                };
                if (g.loop) {
                    for (int64_t c = grp; c < D; c += g.groups) hold(c);
                } else {
                    for (int j = 0; j < g.per; ++j)
                        if ((int64_t)grp * g.per + j < D) hold((int64_t)grp * g.per + j);
                }
            }
        }
    }
    for (int h : held) REQUIRE(h == 1);
}

// The backward's launches: every tile is taken once, a workgroup's partial sums lie inside the workspace, and the
// launch that sums dw of long rows adds every element once to one entry of its chunk.
static void check_bwd_plan(int64_t N, int64_t D, int64_t M, int esz)
{
    const BwdPlan p = norm_bwd_plan(N, D, M, esz);
    REQUIRE(p.blocks >= 1 && p.blocks <= p.g.tiles && p.parts >= 1);
    std::vector<int> taken((size_t)p.g.tiles, 0);
    for (int64_t b = 0; b < p.blocks; ++b)
        for (int64_t i = b; i < p.g.tiles; i += p.blocks) ++taken[(size_t)i];
    for (int t : taken) REQUIRE(t == 1);
    REQUIRE(p.bytes(N, D) >= (size_t)p.parts * D * 8 + (p.apart ? N * 4 : 0));
    if (!p.apart) {
        REQUIRE(p.parts == p.blocks);
        REQUIRE(!p.g.rows || p.g.per * p.g.vec <= 16);  // rows that sum dw in registers
        return;
    }
    REQUIRE(M == 1 && D >= 16 / esz);
    const int V = 16 / esz;
    std::vector<int> cols((size_t)D, 0), rows((size_t)N, 0);
    for (int64_t v = 0; v < p.dw_tiles * kDwThreads; ++v) {
        if (v * V >= D) continue;
        const RowPos q = row_pos((int)v, V, (int)D);
        REQUIRE(q.dup >= 0 && q.dup < V && q.c >= 0 && q.c + V <= D);
        for (int e = q.dup; e < V; ++e) ++cols[(size_t)(q.c + e)];
    }
    for (int64_t k = 0; k < p.parts; ++k) {
        const int64_t lo = k * p.dw_rows, hi = lo + p.dw_rows < N ? lo + p.dw_rows : N;
        REQUIRE(lo < hi);
        for (int64_t r = lo; r < hi; ++r) ++rows[(size_t)r];
    }
    for (int c : cols) REQUIRE(c == 1);
    for (int r : rows) REQUIRE(r == 1);
}

// The launch that adds the parts of dw fits a launch, and its walk takes every column once.
static void check_dw_sum(int64_t D, bool walk)
{
    const int64_t N = 0, M = 0, blocks = dw_sum_blocks(D);
    const int esz = 8;
    REQUIRE(blocks >= 1 && blocks * kDwSumThreads <= (int64_t)UINT32_MAX);
    if (!walk) return;
    std::vector<int> taken((size_t)D, 0);
    for (int64_t b = 0; b < blocks; ++b)
        for (int64_t c0 = b * kDwSumCols; c0 < D; c0 += blocks * kDwSumCols)
            for (int64_t c = c0; c < c0 + kDwSumCols && c < D; ++c) ++taken[(size_t)c];
    for (int t : taken) REQUIRE(t == 1);
}

static void check_dequant(int64_t N, int64_t D, int64_t M, int esz)
{
    const DequantGeom g = dequant_geom(N, D, M, esz);
    const int V = g.vec ? 16 / esz : 1, lanes = 1 << g.lg;
    std::vector<int> held((size_t)(N * D * M), 0);
    for (int64_t b = 0; b < g.blocks; ++b)
        for (int t = 0; t < 256; ++t) {
            const int lane = t & (lanes - 1), grp = t >> g.lg;
            if (M == 1) {
                const int64_t row = b * (256 >> g.lg) + grp;
                if (row >= N) continue;
                for (int v = lane; v < (D + V - 1) / V; v += lanes) {
                    const RowPos p = row_pos(v, V, (int)D);
                    REQUIRE(p.dup >= 0 && p.dup < V && p.c >= 0 && p.c + V <= D);
                    for (int e = p.dup; e < V; ++e) ++held[(size_t)(row * D + p.c + e)];
                }
            } else {
                const int64_t c0 = ((b % g.chunks) * (256 >> g.lg) + grp) * kDequantCpt;
                if (c0 >= D) continue;
                const ColPos p = col_pos(b / g.chunks, lane, V, g.lg, g.tiles_n, N, M);
                REQUIRE(p.n >= 0 && p.n < N && p.m >= 0 && p.m + V <= M && p.dup >= 0);
                for (int j = 0; j < kDequantCpt && c0 + j < D; ++j)
                    for (int e = p.dup; e < V; ++e) ++held[(size_t)((p.n * D + c0 + j) * M + p.m + e)];
            }
        }
    for (int h : held) REQUIRE(h == 1);
}

static void check_xcd()
{
    for (int64_t n = 1; n < 400; ++n) {
        std::vector<int> taken((size_t)n, 0);
        for (int64_t i = 0; i < n; ++i) {
            const int64_t t = xcd_tile(i, n);
            if (t < 0 || t >= n || taken[(size_t)t]++) fail("a tile is taken twice or outside", i, n, t, 0);
        }
    }
}

int main()
{
    check_xcd();
    const int64_t Ds[] = {1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 31, 32, 33, 63, 64, 73, 80, 127, 128, 255, 256, 257, 260, 511, 512, 513,
                          1000, 1024, 1025, 2047, 2048, 2049, 4096, 8191, 8192, 16383, 16384, 16385, 32768, 32769, 70001};
    const int64_t Ms[] = {1, 2, 3, 7, 8, 15, 63, 64, 65, 127, 128, 129, 255, 1000, 1303};
    const int64_t Ns[] = {1, 2, 3, 5, 67, 300};
    int64_t done = 0;
    for (int64_t D : {1, 16, 17, 1 << 20, (1 << 20) + 77, 1 << 23}) check_dw_sum(D, true), ++done;
    for (int64_t D : {(1 << 26) - 15, 1 << 26, 1 << 30}) check_dw_sum(D, false), ++done;
    for (int64_t D : Ds)
        for (int64_t M : Ms)
            for (int64_t N : Ns) {
                if (N * D * M > 600000) continue;
                for (int esz = 2; esz <= 4; esz += 2) {
                    check_norm(N, D, M, esz, false);
                    check_norm(N, D, M, esz, true);
                    check_dequant(N, D, M, esz);
                    check_bwd_plan(N, D, M, esz);
                    done += 4;
                }
            }
    for (int64_t N : {9, 32, 33, 255, 256, 257, 2000, 40001})  // long rows: no walk over the elements
        for (int64_t D : {8192, 8193, 16385, 20000, 32769, 40000, 1 << 20})
            for (int esz = 2; esz <= 4; esz += 2, ++done) check_bwd_plan(N, D, 1, esz);
    printf("%lld geometries checked\n", (long long)done);
    return 0;
}
