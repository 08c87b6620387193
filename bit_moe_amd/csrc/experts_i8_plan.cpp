// Which kernel a product in 8 bits takes.  Host code only.
//
// The 16-bit products' rule, at half the contraction: two codes lie where an
// element lies there, and the matrix cores multiply a register of them in the
// same time.
#include <algorithm>

#include "rows8.h"

namespace bm_host {

namespace {
bool on16(const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0; }
}  // namespace

bool i8_whole(const GemmArgs &g) {
    return on16(g.a.p, g.a.ld) && on16(g.b.p, g.b.ld) && g.K % 16 == 0 && (g.E == 1 || g.b_stride % 16 == 0);
}

GemmPlan i8_plan(const GemmArgs &args, bool whole) {
    GemmArgs g = args;
    g.K = (g.K + 1) / 2;
    return gemm_plan(kForward, g, whole);
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
