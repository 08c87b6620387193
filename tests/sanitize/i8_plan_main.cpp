// Prints what the rule chooses for products in 8 bits (test infrastructure): for
// each line "E R N K whole", the kernel, the parts of the contraction, the few-rows
// kernel's parts and chunks, and 1 where the operands are laid on 16 bytes first.
#include <cstdio>

#include "../../bit_moe_amd/csrc/rows8.h"

int main() {
    using namespace bm_host;
    const char *names[] = {"any", "256x256", "128x256", "128x128", "64x128", "few"};
    int E, R, N, K, whole;
    while (std::scanf("%d %d %d %d %d", &E, &R, &N, &K, &whole) == 5) {
        GemmArgs g{};
        g.E = E;
        g.R = R;
        g.N = N;
        g.K = K;
        const GemmPlan p = i8_plan(g, whole);
        std::printf("%s %d %d %d %d\n", names[p.kind], p.splits, p.parts, p.chunks, (int)p.pack);
    }
    return 0;
}
