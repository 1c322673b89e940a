// bd_fp8_plan.h -- the choice of kernel, tile and K split for the FP8 base products (bd_fp8.hip).
// Host code, plain C++.
#pragma once

#include <stdint.h>

namespace bd {
namespace {

constexpr int kRowsWaves = 8, kRowsMaxT = 64;  // k_fp8_rows: waves a block, its largest batch

// Kernel, tile and K split by a model of their time (us), fitted to measurements at 1..8192
// tokens on 26 sets of matrices, 300 x 8192 to 34816 x 5120 (graph replays on one MI355X).
// Tiles, with n the 128-column stages of a block's K part and `blocks` of them, occ at a time
// on a CU, in rounds of 256 occ (the last of what is left):
//   a + max(sum over rounds of max(b n + e, the round's share of W / 5.9 TB/s),
//           ceil(blocks / 256) (c n + f)) + (S > 1: 3.03 + bytes of the parts / 3.84 TB/s)
// k_fp8_rows: a block's waves go through K in turns of 4096 columns, which wait for memory
// (l + q T each) until the row tiles are so many that all of W's flow takes longer:
//   a + max(turns (l + q T), row tiles K / 4096 (r + p T) + z)
// (2304 x 2304: 4.5 us at 1 token, 6.4 at 24, 10.4 at 64 against 13.0 of the best tile at 96;
// 12288 x 4096: 14.0 at 6 tokens, and at 16 the best tile's 16.1.)
// Against every kernel, tile and split, on eight other sets of matrices and twelve batches, the
// choice is 0.1% off the best on average up to 16 tokens (8% at the worst, 16 tokens on 4096 x
// 11008), 1.4% up to 64 (9%), 0.7% up to 384 (14%) and 0.8% above (5%).
enum { kRows, k256x192, k256x128, k128x256, k128x192, k128x128, k64x128, k128x64, k64x64, k128x32, k64x32 };
struct TileCost {
    int tile, br, bt, occ;
    double a, b, e, c, f;
};
constexpr TileCost kCost[] = {
    {k256x192, 256, 192, 1, 0.243, 1.9, 12.7, 0.03, 16.2},
    {k256x128, 256, 128, 1, 0.558, 1.49, 10.3, 0.58, 4.09},
    {k128x256, 128, 256, 1, 0.653, 1.4, 9.73, 0.537, 1.57},
    {k128x192, 128, 192, 1, 0.119, 1.19, 7.83, 0.246, 0.141},
    {k128x128, 128, 128, 1, 1.13, 0.931, 5.5, 0.104, 0.275},
    {k64x128, 64, 128, 1, 3.86, 0.67, 2.77, 0.084, 0.02},
    {k128x64, 128, 64, 1, 3.04, 0.631, 3.45, 0.059, 0.046},
    {k64x64, 64, 64, 2, 2.76, 0.499, 0.48, 0.341, 1.53},
    {k128x32, 128, 32, 1, 1.03, 0.579, 2.95, 0.044, 0.028},
    {k64x32, 64, 32, 4, 3.58, 0.752, 0.169, 0.189, 0.759}};
struct RowsCost {  // k_fp8_rows<1, 2, 4>
    double a, l, q, r, p, z;
};
constexpr RowsCost kRowsCost[] = {{2.99, 2.01, 0.08, 0.0124, 3.43e-4, 0.59},
                                  {3.36, 2.73, 0.0793, 0.0172, 4.1e-4, 1.04},
                                  {4.0, 3.79, 0.0716, 0.0202, 4.41e-4, 1.54}};
struct Fp8Plan {
    int tile, S;
    int64_t kps;
};
Fp8Plan plan_fp8(int64_t T, int64_t d_in, const int64_t* d_outs, int n, bool split_ok) {
    Fp8Plan pl = {kRows, 1, d_in};
    int64_t N = 0, row_tiles = 0;
    for (int i = 0; i < n; ++i) {
        N += d_outs[i];
        row_tiles += (d_outs[i] + 15) / 16;
    }
    double best = 1e30;
    if (T <= kRowsMaxT) {
        const RowsCost& c = kRowsCost[T <= 16 ? 0 : T <= 32 ? 1 : 2];
        const double units = (double)d_in / (512 * kRowsWaves), turns = units > 1.0 ? (double)((d_in + 512 * kRowsWaves - 1) / (512 * kRowsWaves)) : units;
        const double wait = turns * (c.l + c.q * (double)T), flow = (double)row_tiles * units * (c.r + c.p * (double)T) + c.z;
        best = c.a + (wait > flow ? wait : flow);
    }
    const double stream = (double)(N * d_in) / 5.9e6;
    for (const TileCost& t : kCost) {
        int64_t rt = 0;
        for (int i = 0; i < n; ++i) rt += (d_outs[i] + t.br - 1) / t.br;
        for (int S = 1; S <= (split_ok ? 8 : 1); S *= 2) {
            if (S > 1 && d_in < 1024 * S) break;  // parts of 1024 columns or more
            const int64_t kps = S > 1 ? (d_in + 512 * S - 1) / (512 * S) * 512 : d_in;
            const int64_t parts = (d_in + kps - 1) / kps;
            const int64_t blocks = rt * ((T + t.bt - 1) / t.bt) * parts, hold = 256 * t.occ;
            const int64_t whole = (blocks - 1) / hold;  // rounds before the last
            const double stages = (double)((kps + 127) / 128), one = t.b * stages + t.e;
            const double per = stream / (double)blocks, last = per * (double)(blocks - whole * hold);
            const double full = per * (double)hold > one ? per * (double)hold : one;
            double us = (double)whole * full + (last > one ? last : one);
            const double cu = (double)((blocks + 255) / 256) * (t.c * stages + t.f);
            us = t.a + (us > cu ? us : cu);
            if (parts > 1) us += 3.03 + (double)(T * N * 4 * (parts + 1)) / 3.84e6;
            if (us < best) {
                best = us;
                pl = {t.tile, (int)parts, kps};
            }
        }
    }
    return pl;
}

}  // namespace
}  // namespace bd
