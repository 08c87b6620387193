// Which kernel a 16-bit product takes.  Host code only.
//
// A cost in us for each kernel and each number of parts of the contraction,
// from the sizes the host knows (the groups' own sizes are on the device: they
// are taken as even); the least wins.  Measured in bfloat16, us:
//  one group, N 2048, K 7168     256x256  128x256  128x128  64x128  few rows   parts
//     1 row                         21.0     14.7     13.3    11.3       6.8   of the best 16
//     16                            21.8     15.7     14.4    12.5      12.5   16
//     64                            25.8     20.5     20.8    19.9      34.5   8 (calls, not GPU time, from here on)
//     512                           41.1     32.8     31.6    31.6             4
//     1024                          53.3     43.6     46.0    47.9             4
//     2048                          71.0     65.3     71.1    75.9             2
//     8192                           191      199      221     277             1
//  32 groups of 1024, N 7168, K 2048 879     1014     1182    1543             1
//  256 groups of 8, N 4096, K 7168           2408     2477    2421             1
//  the same, 64 each                3288     2540     2731    3642             1
//  a split: 2048 rows, 128x256: 82.6 whole, 65.3 in 2 parts, 80.0 in 4; weights'
//   gradient of 2048 x 2048 over 8192 rows, 256x256: 155 whole, 75.5 in 4 parts
//  rows not on 16 bytes, which only k_gemm and the few-rows kernel can take
//   (8192 rows): N 2048, K 7168 one element off, forward 358 against 201, rows'
//   gradient 380 and 217, weights' gradient 575 and 195; N 2049, K 7167 in parts
//   1, 2, 4, 8, 16: forward 453 511 578, rows' gradient 474 719, weights'
//   gradient 1314 1104 990 1020 1193; 16 rows forward 119 68 41 28 24 (few rows
//   48), rows' gradient 136 78 50 35; weights' gradient of 4097 x 1023 over 16384
//   rows 2020 1235 800 644 651
#include <algorithm>
#include <cmath>
#include <iterator>

#include "experts.h"

namespace bm_host {

namespace {

bool on16(const void *p, int64_t ld, int cols) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && cols % 8 == 0;
}

struct Shape {
    int kind, bm, bn, slots;    // slots: workgroups a compute unit holds
    double stage, fixed;        // us for 64 of the contraction with every compute unit at work, and per tile
};
const Shape kShapes[] = {
    {kTile256, 256, 256, 1, 1.35, 9.5},
    {kTile128x256, 128, 256, 1, 0.80, 6.0},
    {kTile128, 128, 128, 2, 0.90, 4.0},
    {kTile64x128, 64, 128, 2, 0.60, 4.5},
};
// by layout: its loads wait for one another where rows run along the tile
const Shape kAnyShapes[] = {
    {kAny, 128, 128, 2, 1.15, 5.0},
    {kAny, 128, 128, 2, 3.60, 4.0},
    {kAny, 128, 128, 2, 4.50, 4.0},
};

}  // namespace

void plan_tiles(int layout, const GemmArgs &g, int bm, int bn, GemmPlan *p) {
    p->nt = (g.N + bn - 1) / bn;
    if (layout == kGradWeights) {
        p->mt = (g.M + bm - 1) / bm;
        p->grid = (int64_t)g.E * (((int64_t)p->mt * p->nt * p->splits + 7) / 8) * 8;
    } else {
        p->mt = g.R / bm + std::min(g.E, g.R);
        p->grid = ((int64_t)p->mt * p->nt * p->splits + 7) / 8 * 8;
    }
}

bool gemm_whole(int layout, const GemmArgs &g) {
    if (layout == kGradWeights) return on16(g.a.p, g.a.ld, g.M) && on16(g.b.p, g.b.ld, g.N);
    return on16(g.a.p, g.a.ld, g.K) && on16(g.b.p, g.b.ld, layout == kForward ? g.K : g.N) &&
           (g.E == 1 || g.b_stride % 8 == 0);
}

GemmPlan gemm_plan(int layout, const GemmArgs &g, bool whole) {
    GemmPlan best{};
    double least = 1e30;
    const double cus = cu_count();
    const int groups = std::min(g.E, std::max(g.R, 1));
    const double rows = (double)g.R / groups;             // of a group
    const Shape *const first = whole ? kShapes : kAnyShapes + layout;
    const Shape *const last = whole ? std::end(kShapes) : first + 1;
    for (const Shape *at = first; at < last; at++) {
        const Shape &s = *at;
        if (layout == kGradWeights && s.bm != s.bn) continue;
        // tiles expected: a group's last row tile is half full on average
        const double mt = layout == kGradWeights ? (double)groups * ((g.M + s.bm - 1) / s.bm)
                          : groups == 1          ? (g.R + s.bm - 1) / s.bm
                                                 : groups * std::max(1.0, rows / s.bm + 0.5);
        const double n = mt * ((g.N + s.bn - 1) / s.bn);
        const double k = layout == kGradWeights ? rows : g.K, stages = std::ceil(k / 64);
        const double parts = g.a_low ? 2 : 1;           // (A's two parts one after the other)
        const double out = (double)(layout == kGradWeights ? (double)g.E * g.M : g.R) * g.N;
        for (int splits = 1; splits <= 16; splits *= 2) {
            if (splits > 1 && stages < 4 * splits) break;
            const double rounds = std::ceil(n * splits / (cus * s.slots));
            // parts: written and read in fp32, and a launch with the wait for it
            const double join = splits == 1 ? 0 : 7 + out * 4 * (splits + 1) / 4e6;
            // (a stage takes about three quarters of its time where the GPU is nearly empty)
            const double fill = std::min(1.0, n * splits / (cus * s.slots));
            const double us = rounds * (std::ceil(stages / splits) * parts * s.stage * (0.75 + 0.25 * fill) + s.fixed) + join;
            if (us < least) {
                least = us;
                best.kind = s.kind;
                best.splits = splits;
                best.kper = (int)((stages + splits - 1) / splits) * 64;
                plan_tiles(layout, g, s.bm, s.bn, &best);
                best.ws = splits == 1 ? 0 : ((size_t)out * 4 * splits + 255) / 256 * 256;
            }
        }
    }
    if (layout == kForward) {
        // Few rows: a workgroup reads nb rows of W at 24 bytes a ns and its rows
        // of x, which are in L2, at 44; at 7.5 and 12 where rows are not on 16 bytes
        // (16 rows of 2049 x 7167 in parts 1, 2, 4: 48, 70, 91 us; one of 513 x 7167
        // 28, 17, 12).  The tiles' kernels cannot beat the
        // weights' bytes either.  Over parts 1, 2, 4: one row of 2048 x 7168 10.4,
        // 6.8, 6.8 us, 8 rows 12.6, 8.9, 12.4; one of 512 x 7168 10.2, 6.6, 4.7; one
        // of 16384 x 4096 22.8, 22.1, 23.2, 4 rows 24.2, 26.5, 33.4 (tiles 27.0), 16
        // rows 31.2, 45.8, 76.5 (tiles 27.5).  Groups of more than two rows, of
        // unknown evenness, are the tiles': 8 of 256 experts of 2048 x 2048, one row
        // each 17.4 (tiles 19.2), two 18.5 (19.1), four 28.1 (17.0).
        const double w_rate = whole ? 24e3 : 7.5e3, x_rate = whole ? 44e3 : 12e3;
        least = std::max(least, 5 + (double)groups * g.N * g.K * 2 / 6e6 + (best.splits > 1 ? 7 : 0));
        for (int parts = 1; parts <= 4 && (g.E == 1 || rows <= 2); parts *= 2) {
            const int nb = 16 / parts, chunks = rows <= nb ? 1 : 4, per = nb * chunks;
            const double passes = std::ceil(rows / per), x = std::min(rows, (double)per);
            const double each = std::max(1.0, groups * std::ceil(g.N / (double)nb) * passes / cus);    // of a compute unit
            const double us = 5 + each * g.K * 2 * (nb / w_rate + x / x_rate);
            GemmPlan few{};
            few.kind = kFew;
            few.splits = 1;
            few.parts = parts;
            few.chunks = chunks;
            plan_tiles(layout, g, per, nb, &few);
            if (us < least && few.grid < 1 << 24) {                // (a launch holds less than 2^32 threads)
                least = us;
                best = few;
            }
        }
    }
    if (layout == kGradWeights) best.ws += 2 * (((size_t)g.R * 4 + 255) / 256 * 256);
    return best;
}

size_t gemm_ws_bytes(int layout, const GemmArgs &g) {
    return std::max(gemm_plan(layout, g, true).ws, gemm_plan(layout, g, false).ws);
}

}  // namespace bm_host
