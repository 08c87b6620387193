// Which kernel a product in 8 bits takes.  Host code only.
//
// The kernels are the 16-bit products' (experts_plan.cpp), with two codes where an
// element lies there; their times are not, so the rule is one of its own: a cost
// in us for each kernel and number of parts from the sizes the host knows, the
// least wins.  Measured with bfloat16 outputs, us (calls; a call of the binding
// alone takes 12):
//  one group, N 2048, K 7168     256x256  128x256  128x128  64x128  few rows   parts
//     1 row                                 16.6     15.5    15.5      12.0   of the best 8, 16
//     16                                    17.1     16.4    15.7      12.4   4, 8
//     64                                    19.2     17.7    16.3      17.3   8
//     512                           40.6    31.5     28.7    23.7             4, 4, 2, 1
//     1024                          46.0    37.4     30.7    24.7             4, 4, 1, 1
//     2048                          61.0    42.2     34.3    38.5             4, 1, 1, 1
//     8192                          91.9     109      118     158             1
//  8192 x 4096 x 7168                189     202      210     280             1
//  8192 x 8192 x 8192                391     463      530     688             1
//  32 groups of 1024, N 7168, K 2048 469     592      609     784             1
//  256 groups of 64, N 2048, K 7168  830     685      716     710             1
//  the same, of 43 to 77 rows        827     682      710     840             1
//  the same, 8 each, N 4096                 1229     1254    1227             1
//  8 groups of 1 row, N 4096, K 7168                          44.7     51.9
//  one row, N 16384, K 4096                                   21.6     17.7
//  codes not on 16 bytes, as they lie and laid out anew: 8192 x 2049 x 7167 270, 161; 8
//   groups, 666 rows, 1001 x 2047 33.7 (4 parts), 24.3; 16 x 2049 x 7167 26.4 (16 parts)
#include <algorithm>
#include <cmath>

#include "rows8.h"

namespace bm_host {

namespace {

bool on16(const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0; }

struct Shape {
    int kind, bm, bn, slots;    // slots: workgroups a compute unit holds
    double stage, fixed;        // us for 128 codes of the contraction with every compute unit at work, and per tile
    double alone;               // a stage's share of that where the GPU is nearly empty
};
const Shape kShapes[] = {
    {kTile256, 256, 256, 1, 1.48, 9.5, 0.70},
    {kTile128x256, 128, 256, 1, 0.73, 9.4, 0.70},
    {kTile128, 128, 128, 2, 0.77, 9.4, 0.40},
    {kTile64x128, 64, 128, 2, 0.525, 5.6, 0.45},
};
// (its loads wait for one another: a workgroup alone is slower)
const Shape kAnyShape = {kAny, 128, 128, 2, 1.40, 5.0, 1.4};

}  // namespace

bool i8_whole(const GemmArgs &g) {
    return on16(g.a.p, g.a.ld) && on16(g.b.p, g.b.ld) && g.K % 16 == 0 && (g.E == 1 || g.b_stride % 16 == 0);
}

I8Pack i8_pack(int E, int R, int N, int K) {
    auto up256 = [](size_t n) { return (n + 255) / 256 * 256; };
    I8Pack p{};
    p.ld = (K + 15) / 16 * 16;
    p.x = 0;
    p.scale = up256((size_t)R * p.ld);
    p.w = p.scale + up256((size_t)R * 4);
    p.bytes = p.w + up256((size_t)E * N * p.ld);
    return p;
}

GemmPlan i8_plan(const GemmArgs &g, bool whole) {
    GemmPlan best{};
    double least = 1e30;
    const double cus = cu_count();
    const int groups = std::min(g.E, std::max(g.R, 1));
    const double rows = (double)g.R / groups;             // of a group
    const double stages = std::ceil(g.K / 128.0), out = (double)g.R * g.N;
    const double weights = (double)groups * g.N * g.K;    // bytes
    auto tiles_of = [&](const Shape &s, double before, bool pack) {
        // tiles expected: a group's last row tile is half full on average
        const double mt = groups == 1 ? (g.R + s.bm - 1) / s.bm : groups * std::max(1.0, rows / s.bm + 0.5);
        const double n = mt * ((g.N + s.bn - 1) / s.bn);
        for (int splits = 1; splits <= 16; splits *= 2) {
            if (splits > 1 && stages < 4 * splits) break;
            const double tiles = n * splits, rounds = std::ceil(tiles / (cus * s.slots));
            // parts: written and read in int32, and a launch with the wait for it
            const double join = splits == 1 ? 0 : 7 + out * 4 * (splits + 1) / 4e6;
            // the last round, where it leaves compute units to one workgroup or none
            const double fill = tiles / (cus * s.slots) - (rounds - 1);
            const double last_round = fill <= 0.5 ? s.alone + 0.2 * fill : s.alone + 0.1 + (0.9 - s.alone) * (2 * fill - 1);
            const double work = (rounds - 1 + last_round) * std::ceil(stages / splits) * s.stage + rounds * s.fixed;
            // and no tile takes the weights from memory at more than 40 bytes a ns, all no
            // more than 6000 (5600, 5400 over several rounds); a group's second row tile
            // finds some of them in L2
            const double again = 1 + 0.4 * std::min(mt / groups - 1, 1.0);
            const double rate = rounds <= 1 ? 6e6 : s.bn == 256 ? 5.6e6 : 5.4e6;
            const double us = before + 3 + std::max(work, s.fixed + weights * again / std::min(rate, tiles * 40e3)) + join;
            if (us < least) {
                least = us;
                best.kind = s.kind;
                best.splits = splits;
                best.kper = (int)((stages + splits - 1) / splits) * 64;        // in pairs
                plan_tiles(kForward, g, s.bm, s.bn, &best);
                best.ws = splits == 1 ? 0 : ((size_t)out * 4 * splits + 255) / 256 * 256;
                best.pack = pack;
            }
        }
    };
    if (whole) {
        for (const Shape &s : kShapes) tiles_of(s, 0, false);
    } else {
        tiles_of(kAnyShape, 0, false);
        // Odd K, where the addresses cannot help it: the operands' rows that the
        // product takes laid on 16 bytes first, up to 4 GiB of them
        const size_t packed = i8_pack(g.E, g.R, g.N, g.K).bytes;
        if (g.K % 16 && packed <= (size_t)4 << 30) {
            const double before = 3 + ((double)g.R * g.K + weights) * 2 / 5e6;
            for (const Shape &s : kShapes) tiles_of(s, before, true);
        }
    }
    // Few rows: a workgroup reads nb rows of W at 20 bytes a ns and its rows of x,
    // which are in L2, at 44; at 10 and 5 where rows are not on 16 bytes.  Groups
    // of more than two rows, of unknown evenness, are the tiles'.
    const double w_rate = whole ? 20e3 : 10e3, x_rate = whole ? 44e3 : 5e3;
    for (int parts = 1; parts <= 4 && (g.E == 1 || rows <= 2); parts *= 2) {
        const int nb = 16 / parts, chunks = rows <= nb ? 1 : 4, per = nb * chunks;
        const double passes = std::ceil(rows / per), x = std::min(rows, (double)per);
        const double each = std::max(1.0, groups * std::ceil(g.N / (double)nb) * passes / cus);    // of a compute unit
        const double us = 5 + each * g.K * (nb / w_rate + x / x_rate);
        GemmPlan few{};
        few.kind = kFew;
        few.splits = 1;
        few.parts = parts;
        few.chunks = chunks;
        plan_tiles(kForward, g, per, nb, &few);
        if (us < least && few.grid < 1 << 24) {                // (a launch holds less than 2^32 threads)
            least = us;
            best = few;
        }
    }
    if (best.pack) best.ws += i8_pack(g.E, g.R, g.N, g.K).bytes;
    return best;
}

size_t i8_ws_bytes(int E, int R, int N, int K) {
    GemmArgs g{};
    g.E = E;
    g.R = R;
    g.N = N;
    g.K = K;
    return std::max(i8_plan(g, true).ws, i8_plan(g, false).ws);
}

}  // namespace bm_host
