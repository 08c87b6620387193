// Host sanitizer driver for the 16-bit expert layer's C ABI (test
// infrastructure): its validation (experts.cpp) and the rule that chooses
// kernels, splits and workspaces (experts_plan.cpp), with launcher stand-ins
// that check what they are given and queue nothing.
#include <cstdint>
#include <cstdio>

#include "../../bit_moe_amd/csrc/experts.h"

static int failures = 0, launches = 0;
#define EXPECT(cond)                                                        \
    do {                                                                    \
        if (!(cond)) {                                                      \
            std::printf("FAILED line %d: %s\n", __LINE__, #cond);           \
            failures++;                                                     \
        }                                                                   \
    } while (0)

namespace bm_host {

// the plan covers the product: tiles over all rows and columns, parts over
// the whole contraction, workspace for every part
int launch_gemm(int layout, int, const GemmArgs &g, void *, hipStream_t) {
    launches++;
    for (int whole = 0; whole < 2; whole++) {
        const GemmPlan p = gemm_plan(layout, g, whole);
        const bool few = p.kind == kFew;
        const int bm = few ? 16 / p.parts * p.chunks : p.kind == kTile256 ? 256 : p.kind == kTile64x128 ? 64 : 128;
        const int bn = few ? 16 / p.parts : p.kind == kTile256 || p.kind == kTile128x256 ? 256 : 128;
        EXPECT(whole || few || p.kind == kAny);
        EXPECT(!few || (layout == kForward && p.splits == 1 && (p.chunks == 1 || p.chunks == 4) &&
                        (p.parts == 1 || p.parts == 2 || p.parts == 4) && p.grid * 256 < (int64_t)1 << 32));
        EXPECT(layout != kGradWeights || p.kind == kAny || p.kind == kTile256 || p.kind == kTile128);
        EXPECT(p.splits >= 1 && (int64_t)p.nt * bn >= g.N && (int64_t)(p.nt - 1) * bn < g.N);
        const int64_t n = (int64_t)p.mt * p.nt * p.splits;
        if (layout == kGradWeights) {
            EXPECT((int64_t)p.mt * bm >= g.M && p.grid >= n * g.E && p.grid % 8 == 0);
            EXPECT(p.ws >= (p.splits > 1 ? (size_t)p.splits * g.E * g.M * g.N * 4 : 0) + (size_t)g.R * 8);
        } else {
            // row tiles of any groups of R rows: a part of a tile for each group that has rows
            EXPECT((int64_t)p.mt * bm >= g.R && p.mt >= g.R / bm + (g.E < g.R ? g.E : g.R) && p.grid >= n);
            EXPECT(p.splits == 1 || (int64_t)p.splits * p.kper >= g.K);
            EXPECT(p.splits == 1 || p.ws >= (size_t)p.splits * g.R * g.N * 4);
        }
        EXPECT(p.ws <= gemm_ws_bytes(layout, g) && p.ws % 256 == 0);
    }
    // the maps' division by multiplication
    for (const GemmRows *q : {&g.a, &g.b, &g.c})
        if (q->map && q->mul)
            for (uint32_t x : {0u, 1u, 6u, 7u, 8u, 9u, 1000003u, 0x7FFFFFFEu, 0x7FFFFFFFu})
                EXPECT((uint32_t)(((uint64_t)x * q->mul) >> 32) >> q->shift == x / (uint32_t)((intptr_t)q->p / 2));
    return BITMOE_EHIP;
}
int act_backward_slices(int T, int N) { return T / 16 + 1 + N / (1 << 18); }
int launch_act_backward(const ActBackward &, int, hipStream_t) { return BITMOE_OK; }
int launch_swiglu(const bitmoe_rows &, const bitmoe_rows &, const bitmoe_rows &, int, hipStream_t) { return BITMOE_EHIP; }
int launch_swiglu_backward(const bitmoe_rows &, const bitmoe_rows &, const bitmoe_rows &, const bitmoe_rows &,
                           const bitmoe_rows &, int, hipStream_t) {
    return BITMOE_EHIP;
}
int launch_combine(const bitmoe_rows &, const float *, int, int, const bitmoe_rows *, const bitmoe_rows &, hipStream_t) {
    return BITMOE_EHIP;
}
int launch_combine_backward(const bitmoe_rows &, const bitmoe_rows *, const float *, int, int, const bitmoe_rows *,
                            float *, int, hipStream_t) {
    return BITMOE_EHIP;
}

}  // namespace bm_host

static void *at(uintptr_t a) { return reinterpret_cast<void *>(a); }
static bitmoe_rows rows(int n, int cols, int64_t ld = 0, int dtype = BITMOE_BF16) {
    return bitmoe_rows{at(1 << 20), nullptr, ld ? ld : cols, n, cols, 1, dtype};
}
static bitmoe_experts experts(int E, int N, int K, int dtype = BITMOE_BF16) {
    return bitmoe_experts{at(2 << 20), K, (int64_t)N * K, E, N, K, dtype};
}

int main() {
    const int32_t *ints = static_cast<const int32_t *>(at(3 << 20));
    void *ws = at(4 << 20);
    const size_t lots = ~(size_t)0 >> 1;
    for (int E : {1, 2, 7, 32, 256, 1024})
        for (int R : {1, 3, 64, 129, 5000, 65536, 1 << 24})
            for (int N : {1, 8, 100, 2048, 7168, 1 << 18})
                for (int K : {1, 64, 1001, 7168, 1 << 18}) {
                    const bitmoe_experts w = experts(E, N, K);
                    const bitmoe_rows x = rows(R, K), y = rows(R, N, 0, BITMOE_F32), dy = rows(R, N);
                    EXPECT(moe_expert_matmul(&x, &w, ints, R, &y, ws, lots, nullptr) == BITMOE_EHIP);
                    EXPECT(moe_expert_matmul_dx(&dy, &w, ints, R, &x, ws, lots, nullptr) == BITMOE_EHIP);
                    EXPECT(moe_expert_matmul_dw(&dy, &x, ints, R, &w, 0, ws, lots, nullptr) == BITMOE_EHIP);
                    const size_t need = moe_expert_matmul_workspace_bytes(BITMOE_MATMUL_DW, E, R, N, K);
                    EXPECT(need > 0 && need % 256 == 0);
                    EXPECT(moe_expert_matmul_dw(&dy, &x, ints, R, &w, 0, ws, need, nullptr) == BITMOE_EHIP);
                    EXPECT(moe_expert_matmul_dw(&dy, &x, ints, R, &w, 0, ws, need - 1, nullptr) == BITMOE_EWORKSPACE);
                    if (E == 1) {
                        const size_t lin = moe_linear_workspace_bytes(R, N, K);
                        const size_t back = moe_linear_backward_workspace_bytes(R, N, K);
                        EXPECT(moe_linear(&x, &w, nullptr, 2, &y, &dy, &y, ws, lin, nullptr) == BITMOE_EHIP);
                        EXPECT(moe_linear_backward(&dy, &x, &w, 2, &dy, &x, &w, ws, 0, ws, back, nullptr) == BITMOE_EHIP);
                        EXPECT(moe_linear_backward(&dy, &x, &w, 2, &dy, &x, &w, ws, 0, ws, back - 1, nullptr) ==
                               BITMOE_EWORKSPACE);
                    }
                }
    // maps, their divisors (the stand-in finds the divisor in the data pointer, half of it)
    for (int d : {1, 2, 3, 7, 8, 1000, 65537, 0x7FFFFFFF}) {
        const bitmoe_experts w = experts(4, 16, 16);
        bitmoe_rows x = rows(8, 16);
        x.map = ints;
        x.div = d;
        x.data = at((uintptr_t)d * 2);
        EXPECT(moe_expert_matmul(&x, &w, ints, 8, &x, ws, lots, nullptr) == BITMOE_EHIP);
    }
    EXPECT(launches > 2000);
    const bitmoe_rows o = rows(32, 100), t = rows(4, 100);
    const float *fw = static_cast<const float *>(at(5 << 20));
    EXPECT(moe_swiglu(&o, &o, &o, nullptr) == BITMOE_EHIP);
    EXPECT(moe_swiglu_backward(&o, &o, &o, &o, &o, nullptr) == BITMOE_EHIP);
    EXPECT(moe_combine(&o, fw, 4, 8, &t, &t, nullptr) == BITMOE_EHIP);
    EXPECT(moe_combine_backward(&t, &o, fw, 4, 8, &o, const_cast<float *>(fw), nullptr) == BITMOE_EHIP);
    std::printf(failures ? "experts sanitizer driver: %d check(s) failed\n" : "experts sanitizer driver: ok\n", failures);
    return failures ? 1 : 0;
}
