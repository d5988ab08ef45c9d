// linear_check.cpp — replays the index arithmetic of the 8-bit form and the channel products on the CPU.
//
//   linear_check          (built by the tests with g++ and the address and undefined-behaviour sanitizers)
//
// Walks the form's writer and reader as the kernels do, for many shapes and element sizes (every access inside its tensor,
// every element and code met, the LDS indexes inside what a launch asks for, a tile's codes read where they were written),
// and checks the division by a product, the products' LDS layouts, the ring of the kernels that hold their weights in registers
// (direct loads and the reads of a tile), the map of workgroups to tiles and the splits of the weight's gradient.  Prints the
// number of geometries checked.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "linear_plan.hpp"

using namespace disco;

static void fail(const char *what, int64_t a, int64_t b, int64_t c, int d)
{
    printf("FAILED: %s at %lld, %lld, %lld, %d\n", what, (long long)a, (long long)b, (long long)c, d);
    exit(1);
}

#define REQUIRE(x) do { if (!(x)) fail(#x, N, D, M, esz); } while (0)

static void check_form(int64_t N, int64_t D, int64_t M, int esz)
{
    const FormGeom g = form_geom(N, D, M, esz);
    const int64_t Dp = padded_channels(D), P = N * M;
    const int nv = (int)(Dp / kFormChannels), lanes = 1 << g.lg;
    REQUIRE(Dp % 16 == 0 && Dp >= D && Dp < D + 16);
    REQUIRE(g.threads >= 64 && g.threads <= kNormMaxThreads && g.threads % 64 == 0 && g.tiles >= 1);
    REQUIRE(form_lds_bytes(g, Dp) <= 65 * 1024);
    std::vector<int> codes((size_t)(P * nv), 0), held((size_t)(N * D * M), 0);
    if (g.loop) {
        const int groups = g.threads >> g.lg;
        REQUIRE(form_lds_bytes(g, Dp) >= (size_t)2 * lanes * 4 && groups * lanes == g.threads && g.vec == 1);
        for (int64_t tile = 0; tile < g.tiles; ++tile)
            for (int t = 0; t < g.threads; ++t) {
                const ColPos p = col_pos(tile, t & (lanes - 1), 1, g.lg, 1, N, M);
                REQUIRE(p.n >= 0 && p.n < N && p.m >= 0 && p.m < M);
                for (int64_t c = (int64_t)(t >> g.lg) * 8; c < Dp; c += (int64_t)groups * 8) {
                    REQUIRE(c + 8 <= Dp);
                    if (!p.dup) ++codes[(size_t)((p.n * M + p.m) * nv + c / 8)];
                    for (int64_t j = c; j < c + 8 && j < D; ++j)
                        if (!p.dup) ++held[(size_t)((p.n * D + j) * M + p.m)];
                }
            }
    } else if (g.rows) {
        REQUIRE(M == 1 && g.slots * lanes == g.threads && (int64_t)g.per * lanes >= nv);
        for (int64_t tile = 0; tile < g.tiles; ++tile)
            for (int t = 0; t < g.threads; ++t) {
                const int64_t want = tile * g.slots + (t >> g.lg), row = want < N ? want : N - 1;
                for (int k = 0; k < g.per; ++k) {
                    const int64_t c = (int64_t)(k * lanes + (t & (lanes - 1))) * 8;
                    if (c < Dp && want < N) ++codes[(size_t)(row * nv + c / 8)];
                    for (int64_t j = c; j < c + 8 && j < D; ++j)
                        if (want < N) ++held[(size_t)(row * D + j)];
                }
            }
    } else {
        const int PT = lanes * g.vec, half = nv / 2;
        REQUIRE(g.slots == nv && g.threads >= nv * lanes && form_lds_bytes(g, Dp) == (size_t)PT * Dp + (size_t)PT * 8);
        const FastDiv by = fast_div((uint32_t)half);
        for (int64_t tile = 0; tile < g.tiles; ++tile) {
            std::vector<int64_t> lds((size_t)PT * nv, -1);   // which code (point, eight) lies there
            for (int t = 0; t < g.threads; ++t) {
                const int lane = t & (lanes - 1), grp = t >> g.lg;
                const ColPos p = col_pos(tile, lane, g.vec, g.lg, g.tiles_n, N, M);
                REQUIRE(p.n >= 0 && p.n < N && p.m >= 0 && p.m + g.vec <= M && p.dup >= 0);
                if (grp >= nv) continue;
                int cg = grp + lane % nv;
                if (cg >= nv) cg -= nv;
                for (int e = 0; e < g.vec; ++e) {
                    const int at = (lane * g.vec + e) * nv + cg;
                    REQUIRE(at * 8 == form_lds(lane * g.vec + e, grp, nv, lane) && at < PT * nv && lds[at] < 0);
                    lds[at] = (p.n * M + p.m + e) * nv + grp;
                    for (int j = grp * 8; j < grp * 8 + 8 && j < D; ++j)
                        if (e >= p.dup) ++held[(size_t)((p.n * D + j) * M + p.m + e)];
                }
            }
            for (int i = 0; i < PT * half; ++i) {
                const int pt = (int)by.div(i), h = i - pt * half, l = pt / g.vec;
                const ColPos at = col_pos(tile, l, g.vec, g.lg, g.tiles_n, N, M);
                const int64_t point = at.n * M + at.m + (pt - l * g.vec);
                for (int k = 0; k < 2; ++k) {
                    const int64_t code = lds[(size_t)form_lds(pt, 2 * h + k, nv, l) / 8];
                    REQUIRE(code == point * nv + 2 * h + k);
                    if (pt - l * g.vec >= at.dup) ++codes[(size_t)code];
                }
            }
        }
    }
    for (int v : codes) REQUIRE(v == 1);
    for (int v : held) REQUIRE(v == 1);
}

template <int N>
static void check_across()
{
    std::vector<int> used(64 * N * 2 / 16, 0);
    for (int r = 0; r < 64; ++r)
        for (int n = 0; n < N; n += 8) {
            const int at = bwd_across<N>(r, n);
            if (at % 16 || at < 0 || at + 16 > 64 * N * 2 || used[at / 16]++) fail("across", N, r, n, 0);
            for (int e = 0; e < 8; e += 4)  // what a transposing read takes: four elements
                if (bwd_across<N>(r, n + e) != at + 2 * e) fail("across within a piece", N, r, n, e);
        }
}

// Slot s is written by a direct load, read by row and piece; sixteen rows' equal pieces meet each bank (of 4 bytes, 64 of
// them) once.
template <int K>
static void check_slots(int rows)
{
    for (int s = 0; s < rows * K / 16; ++s)
        if (lin_at<K>(s / (K / 16), lin_piece<K>(s)) != 16 * s || lin_piece<K>(s) >= K / 16) fail("slot", rows, s, K, 0);
    for (int r = 0; r < rows; r += 16)
        for (int p = 0; p < K / 16; ++p) {
            int banks = 0;
            for (int i = 0; i < 16; ++i) banks |= 1 << (lin_at<K>(r + i, p) / 16 % 16);
            if (banks != 0xffff) fail("banks", r, p, K, 0);
        }
}

// One stage of a ring: what each 16 bytes hold, by the direct loads (instruction i of 256 threads writes slots 256 i ..), as
// point << 20 | first byte of the point's run; -1: nothing.
struct Stage {
    std::vector<int64_t> at;
    int64_t size;
    explicit Stage(int bytes) : at((size_t)bytes / 16, -1), size(bytes) {}
    template <int K>
    void load(int base, int loads, int points, const char *what)
    {
        for (int i = 0; i < loads; ++i)
            for (int tid = 0; tid < 256; ++tid) {
                const int s = i * 256 + tid, row = s / (K / 16), lds = base + 16 * (i * 256 + (tid >> 6) * 64) + 16 * (tid & 63);
                if (lds + 16 > size || at[(size_t)lds / 16] >= 0 || row >= points) fail(what, s, row, lds, K);
                at[(size_t)lds / 16] = (int64_t)row << 20 | 16 * lin_piece<K>(s);
            }
    }
    // n bytes at `lds` are the bytes `byte` .. of point `p`
    void read(int64_t lds, int n, int p, int byte, const char *what) const
    {
        if (lds < 0 || lds % n || lds + n > size || at[(size_t)lds / 16] != ((int64_t)p << 20 | (byte & ~15)) || lds % 16 != byte % 16) fail(what, lds, p, byte, n);
    }
    // the four waves' copies of the scales: 64 lanes of 4 bytes each, behind all else
    void scales(int base, int points)
    {
        for (int w = 0; w < 4; ++w) {
            for (int b = 0; b < 256; b += 16)
                if (base + 256 * w + b + 16 > size || at[(size_t)(base + 256 * w + b) / 16] >= 0) fail("scales", base, w, b, 0);
                else at[(size_t)(base + 256 * w + b) / 16] = -2 - w;
            if (4 * points > 256) fail("scales of a tile", points, w, 0, 0);
        }
        if (base + 4 * 256 != size) fail("stage", base, (int)size, 0, 0);
    }
};

// A full tile of the product: whole rows of K bytes, then the reads of its operands.
template <int K>
static int check_stay()
{
    typedef LStay<K> L;
    Stage st(L::kStage);
    st.load<K>(0, L::LOADS - 1, L::PT, "product's tile");
    st.scales(L::kTile, L::PT);
    for (int j = 0; j < L::PT; j += 32)
        for (int k = 0; k < K / 32; ++k)
            for (int lane = 0; lane < 64; ++lane) st.read(lin_at<K>(j + (lane & 31), 2 * k + (lane >> 5)), 16, j + (lane & 31), 32 * k + 16 * (lane >> 5), "product's operand");
    if (2 * (L::RING * L::kStage + 2 * kStayChannels * 4) > 160 * 1024) fail("two workgroups' LDS", K, L::RING, L::kStage, 0);
    return 1;
}

// And of the input's gradient, with the checkpoint of a lane's four neighbouring channels.
template <int KB, bool KEPT>
static int check_bwd_stay()
{
    typedef GStay<KB, KEPT> L;
    Stage st(L::kStage);
    st.load<KB>(0, L::LOADS, L::PT, "gradient's tile");
    if (KEPT) {
        // (a byte of the checkpoint is told from one of the gradients by its point: 32 points or 64 further on)
        Stage kt(L::kKept);
        kt.load<L::CB>(0, L::KLOADS, L::PT, "checkpoint's tile");
        for (int64_t i = 0; i < (int64_t)kt.at.size(); ++i) {
            if (st.at[(size_t)(L::kTile / 16 + i)] >= 0 || kt.at[(size_t)i] < 0) fail("checkpoint's place", i, KB, 0, 0);
            st.at[(size_t)(L::kTile / 16 + i)] = kt.at[(size_t)i] + ((int64_t)L::PT << 20);
        }
        st.scales(L::kTile + L::kKept, L::PT);
    }
    for (int j = 0; j < L::PT; j += 32)
        for (int lane = 0; lane < 64; ++lane) {
            const int r = lane & 31, h = lane >> 5;
            for (int k = 0; k < KB / 32; ++k) st.read(lin_at<KB>(j + r, 2 * k + h), 16, j + r, 32 * k + 16 * h, "gradient's operand");
            for (int wave = 0; KEPT && wave < 4; ++wave)
                for (int i = 0; i < L::FW; ++i)
                    for (int g = 0; g < 4; ++g) {
                        const int col = L::CW * wave + 32 * i + 8 * g + 4 * h;
                        st.read(L::kTile + lin_at<L::CB>(j + r, col >> 4) + (col & 15), 4, L::PT + j + r, col, "checkpoint");
                    }
        }
    for (int64_t v : st.at)
        if (v == -1) fail("a place of the stage that nothing fills", KB, KEPT, 0, 0);
    if (2 * L::RING * L::kStage > 160 * 1024) fail("two workgroups' LDS", KB, L::RING, L::kStage, KEPT);
    return 1;
}

int main()
{
    int n = 0;
    for (int64_t d : {1, 2, 3, 5, 7, 11, 64, 181, 360, 1000, 16471, 65535, 65536, 65537, 1038240, 2076480, (1 << 30) - 1, 1 << 30, 2147479552}) {
        const FastDiv f = fast_div((uint32_t)d);
        for (int64_t q = 0; q <= kMaxPoints / d; q += 1 + kMaxPoints / d / 5000)
            for (int64_t k : {(int64_t)-1, (int64_t)0, (int64_t)1, d / 2, d - 1}) {
                const int64_t v = q * d + k;
                if (v >= 0 && v < ((int64_t)1 << 31) && f.div((uint32_t)v) != v / d) fail("division", v, d, 0, 0);
            }
        ++n;
    }
    for (int esz : {2, 4}) {
        for (int64_t N : {1, 2, 5, 17})
            for (int64_t D : {1, 8, 16, 17, 33, 80, 130, 256, 511, 600, 1030})
                for (int64_t M : {1, 2, 5, 35, 63, 64, 65, 117, 260, 1031}) {
                    check_form(N, D, M, esz);
                    ++n;
                }
        for (int64_t D : {1024, 1025, 2032, 2047, 2048, 2049, 4097, 8192, 16385, 32768, 32769, 40000}) {
            check_form(3, D, 1, esz);
            check_form(1, D, 70, esz);
            check_form(2, D, 5, esz);
            n += 3;
        }
    }
    check_form(700, 256, 1, 2);
    check_form(1, 64, 66000, 2);  // tiles of the whole run
    check_across<32>();
    check_across<128>();
    check_across<256>();
    for (int rows : {128, 256}) {
        check_slots<64>(rows);
        check_slots<128>(rows);
        check_slots<256>(rows);
        check_slots<512>(rows);
    }
    check_slots<1024>(32);
    n += check_stay<64>() + check_stay<128>() + check_stay<256>() + check_stay<512>();
    n += check_bwd_stay<128, false>() + check_bwd_stay<256, false>() + check_bwd_stay<512, false>() + check_bwd_stay<1024, false>();
    n += check_bwd_stay<128, true>() + check_bwd_stay<256, true>() + check_bwd_stay<512, true>() + check_bwd_stay<1024, true>();
    for (int64_t total : {1, 7, 8, 9, 255, 256, 1000, 8104}) {
        std::vector<int> met((size_t)total, 0);
        for (int64_t i = 0; i < total; ++i) {
            for (int32_t fast : {1, 3, 8}) {
                int32_t a, b;
                lin_tile(i, total, fast, &a, &b);
                if (a < 0 || a >= fast || b < 0) fail("tile", total, i, fast, 0);
                if (fast == 3 && (int64_t)b * 3 + a < total) ++met[(size_t)b * 3 + a];
            }
        }
        for (int v : met)
            if (v != 1) fail("tile met", total, v, 0, 0);
    }
    for (int64_t P : {(int64_t)1, (int64_t)63, (int64_t)64, (int64_t)65, (int64_t)1000, (int64_t)16400, (int64_t)70000, (int64_t)259200, (int64_t)2076480, kMaxPoints})
        for (int64_t C : {1, 32, 33, 128, 129, 256, 512, 2048, 8192})
            for (int64_t Co : {1, 73, 129, 256, 2048, 8192}) {
                const WeightPlan p = weight_plan(P, C, Co);
                const int64_t all = ceil_div64(P, 64);
                // every split has a step, and all steps have a split; a split's first point fits 32 bits
                if (p.splits < 1 || p.steps < 1 || (int64_t)(p.splits - 1) * p.steps >= all || (int64_t)p.splits * p.steps < all ||
                    (int64_t)p.splits * p.steps * 64 > ((int64_t)1 << 32)) fail("splits", P, C, Co, p.splits);
                if (weight_bytes(p, C, Co, true) != (p.splits == 1 ? 0 : (size_t)p.splits * (Co * C + Co * p.nx) * 4)) fail("bytes", P, C, Co, 0);
                ++n;
            }
    printf("%d geometries checked\n", n);
    return 0;
}
