// Prints the kernel that each product read from stdin takes (test
// infrastructure): lines "layout E R N K whole low" to "kind splits parts
// chunks".  N and K: the product's columns and contraction (weights' gradient:
// its rows, columns).  Host code only.
#include <cstdio>

#include "../../bit_moe_amd/csrc/experts.h"

int main() {
    using namespace bm_host;
    static const char *const kinds[] = {"any", "256x256", "128x256", "128x128", "64x128", "few"};
    int layout, E, R, N, K, whole, low;
    while (std::scanf("%d %d %d %d %d %d %d", &layout, &E, &R, &N, &K, &whole, &low) == 7) {
        GemmArgs g{};
        g.E = E;
        g.R = R;
        g.M = N;
        g.N = layout == kGradWeights ? K : N;
        g.K = K;
        g.a_low = low;
        const GemmPlan p = gemm_plan(layout, g, whole != 0);
        std::printf("%s %d %d %d\n", kinds[p.kind], p.splits, p.parts, p.chunks);
    }
    return 0;
}
