// Which kernel a 16-bit product takes.  Host code only.
#include <algorithm>
#include <cmath>

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

void tiles(int layout, const GemmArgs &g, int bm, int bn, GemmPlan *p) {
    p->nt = (g.N + bn - 1) / bn;
    if (layout == kGradWeights) {
        p->mt = (g.M + bm - 1) / bm;
        p->grid = (int64_t)g.E * (((int64_t)p->mt * p->nt * p->splits + 7) / 8) * 8;
    } else {
        p->mt = g.R / bm + std::min(g.E, g.R);
        p->grid = ((int64_t)p->mt * p->nt * p->splits + 7) / 8 * 8;
    }
}

}  // namespace

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
    for (const Shape &s : kShapes) {
        if (whole ? layout == kGradWeights && s.bm != s.bn : s.kind != kTile128) continue;
        // tiles expected: a group's last row tile is half full on average
        const double mt = layout == kGradWeights ? (double)groups * ((g.M + s.bm - 1) / s.bm)
                          : groups == 1          ? (g.R + s.bm - 1) / s.bm
                                                 : groups * std::max(1.0, rows / s.bm + 0.5);
        const double n = mt * ((g.N + s.bn - 1) / s.bn);
        const double k = layout == kGradWeights ? rows : g.K, stages = std::ceil(k / 64);
        const double out = (double)(layout == kGradWeights ? (double)g.E * g.M : g.R) * g.N;
        for (int splits = 1; splits <= 16; splits *= 2) {
            if (splits > 1 && stages < 4 * splits) break;
            const double rounds = std::ceil(n * splits / (cus * s.slots));
            // parts: written and read in fp32, and a launch with the wait for it
            const double join = splits == 1 ? 0 : 7 + out * 4 * (splits + 1) / 4e6;
            // (a stage takes about three quarters of its time where the GPU is nearly empty)
            const double fill = std::min(1.0, n * splits / (cus * s.slots));
            const double us = rounds * (std::ceil(stages / splits) * s.stage * (0.75 + 0.25 * fill) + s.fixed) + join;
            if (us < least) {
                least = us;
                best.kind = whole ? s.kind : kAny;
                best.splits = splits;
                best.kper = (int)((stages + splits - 1) / splits) * 64;
                tiles(layout, g, s.bm, s.bn, &best);
                best.ws = splits == 1 ? 0 : ((size_t)out * 4 * splits + 255) / 256 * 256;
            }
        }
    }
    if (layout == kForward) {
        // few rows: bound by the weights, read once per pass of up to 16 rows /
        // parts * chunks of a group, and by x, read by every workgroup (from
        // L2); one launch
        int parts = 1;
        while (parts < 4 && groups * std::ceil(g.N * parts / 16.0) < 2 * cus) parts *= 2;
        const int nb = 16 / parts, chunks = g.R <= nb ? 1 : 4, per = nb * chunks;
        const double nt = std::ceil(g.N / (double)nb), passes = std::max(1.0, rows / per);
        const double us = 4 + groups * nt * nb * g.K * 2 * passes / 4.5e6 + (double)g.R * g.K * 2 * nt / 8e6;
        GemmPlan few{};
        few.kind = kFew;
        few.splits = 1;
        few.parts = parts;
        few.chunks = chunks;
        tiles(layout, g, per, nb, &few);
        if (us < least && few.grid < 1 << 24) best = few;          // (a launch holds less than 2^32 threads)
    }
    if (layout == kGradWeights) best.ws += 2 * (((size_t)g.R * 4 + 255) / 256 * 256);
    return best;
}

size_t gemm_ws_bytes(int layout, const GemmArgs &g) {
    return std::max(gemm_plan(layout, g, true).ws, gemm_plan(layout, g, false).ws);
}

}  // namespace bm_host
