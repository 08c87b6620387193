// Host sanitizer driver for the C ABI in 8 bits and of the block norms (test
// infrastructure): its validation (rows8.cpp, norm.cpp) and the rule that chooses
// kernels, parts and workspaces (experts_i8_plan.cpp), with launcher stand-ins that
// check what they are given and queue nothing.
#include <cstdint>
#include <cstdio>

#include "../../bit_moe_amd/csrc/norm.h"
#include "../../bit_moe_amd/csrc/rows8.h"

static int failures = 0, launches = 0;
#define EXPECT(cond)                                                        \
    do {                                                                    \
        if (!(cond)) {                                                      \
            std::printf("FAILED line %d: %s\n", __LINE__, #cond);           \
            failures++;                                                     \
        }                                                                   \
    } while (0)

namespace bm_host {

// the plan covers the product: tiles over all rows and columns, parts over the whole
// contraction, workspace for every part and for what is laid out
int launch_gemm_i8(int, const GemmArgs &g, void *, hipStream_t) {
    launches++;
    for (int whole = 0; whole < 2; whole++) {
        const GemmPlan p = i8_plan(g, whole);
        const bool few = p.kind == kFew;
        const int bm = few ? 16 / p.parts * p.chunks : p.kind == kTile256 ? 256 : p.kind == kTile64x128 ? 64 : 128;
        const int bn = few ? 16 / p.parts : p.kind == kTile256 || p.kind == kTile128x256 ? 256 : 128;
        EXPECT(whole || few || p.pack || p.kind == kAny);
        EXPECT(!p.pack || (!whole && g.K % 16 != 0 && !few && p.kind != kAny));
        EXPECT(!few || (p.splits == 1 && (p.chunks == 1 || p.chunks == 4) &&
                        (p.parts == 1 || p.parts == 2 || p.parts == 4) && p.grid * 256 < (int64_t)1 << 32));
        EXPECT(p.splits >= 1 && (int64_t)p.nt * bn >= g.N && (int64_t)(p.nt - 1) * bn < g.N);
        EXPECT((int64_t)p.mt * bm >= g.R && p.mt >= g.R / bm + (g.E < g.R ? g.E : g.R) && p.grid >= (int64_t)p.mt * p.nt * p.splits);
        EXPECT(p.splits == 1 || (int64_t)p.splits * p.kper * 2 >= g.K);
        const I8Pack k = i8_pack(g.E, g.R, g.N, g.K);
        EXPECT(k.ld % 16 == 0 && k.ld >= g.K && k.scale >= (size_t)g.R * k.ld && k.w >= k.scale + (size_t)g.R * 4 &&
               k.bytes >= k.w + (size_t)g.E * g.N * k.ld && (k.x | k.scale | k.w | k.bytes) % 256 == 0);
        EXPECT(p.ws >= (p.splits > 1 ? (size_t)p.splits * g.R * g.N * 4 : 0) + (p.pack ? k.bytes : 0));
        EXPECT(p.ws <= i8_ws_bytes(g.E, g.R, g.N, g.K) && p.ws % 256 == 0);
    }
    return BITMOE_EHIP;
}
int launch_quantize_rows(const bitmoe_rows &, const bitmoe_rows8 &, hipStream_t) { return BITMOE_EHIP; }
int launch_dequantize_rows(const bitmoe_rows8 &, const bitmoe_rows &, hipStream_t) { return BITMOE_EHIP; }
int launch_swiglu_rows8(const bitmoe_rows &, const bitmoe_rows &, const bitmoe_rows8 &, hipStream_t) { return BITMOE_EHIP; }
int launch_swiglu_checkpoint(const bitmoe_rows &, const bitmoe_rows &, const bitmoe_rows &, const bitmoe_rows8 &,
                             const bitmoe_rows8 &, hipStream_t) {
    return BITMOE_EHIP;
}
int launch_swiglu_checkpoint_backward(const bitmoe_rows &, const bitmoe_rows8 &, const bitmoe_rows8 &, const bitmoe_rows &,
                                      const bitmoe_rows &, const bitmoe_rows *, hipStream_t) {
    return BITMOE_EHIP;
}
int launch_block_norm(const NormArgs &a, int, hipStream_t) {
    EXPECT(a.T > 0 && (a.gate.ld == 0 || a.gate.ld >= a.H));
    return BITMOE_EHIP;
}
int launch_block_norm_backward(const NormBackArgs &a, int, hipStream_t) {
    const NormShape b = norm_shape(a.T, a.H);
    // the threads of a row hold it; every row has a place
    EXPECT((int64_t)b.nt * b.pieces * 8 >= a.H && b.nt % 64 == 0 && b.nt * b.groups <= 1024 && b.groups >= 1);
    EXPECT(b.pieces == 1 ? b.nt * b.groups <= 256 : b.nt <= 512 ? b.nt * b.groups <= 512 : a.H > 8192);
    EXPECT((b.slices == 0) == (a.T == 0) && (int64_t)b.slices * b.groups <= (int64_t)a.T + b.groups - 1);
    return BITMOE_EHIP;
}

}  // namespace bm_host

static void *at(uintptr_t a) { return reinterpret_cast<void *>(a); }
static bitmoe_rows rows(int n, int cols, int dtype = BITMOE_BF16) {
    return bitmoe_rows{at(1 << 20), nullptr, cols, n, cols, 1, dtype};
}
static bitmoe_rows8 rows8(int n, int cols, int block = 0) {
    return bitmoe_rows8{rows(n, cols, BITMOE_I8), static_cast<float *>(at(6 << 20)), bm_host::row_blocks(cols, block), block, 0};
}

int main() {
    const int32_t *ints = static_cast<const int32_t *>(at(3 << 20));
    void *ws = at(4 << 20);
    const size_t lots = ~(size_t)0 >> 1;
    for (int E : {1, 2, 7, 32, 256, 1024})
        for (int R : {1, 3, 64, 129, 5000, 65536, 1 << 24})
            for (int N : {1, 8, 100, 2048, 7168, 1 << 18})
                for (int K : {1, 64, 1001, 7168, 7169, (1 << 17) - 1}) {
                    const bitmoe_experts8 w{{at(2 << 20), K, (int64_t)N * K, E, N, K, BITMOE_I8}, static_cast<float *>(at(5 << 20)), N};
                    const bitmoe_rows8 x = rows8(R, K);
                    const bitmoe_rows y = rows(R, N, BITMOE_F32);
                    EXPECT(moe_expert_matmul_i8(&x, &w, ints, R, &y, ws, lots, nullptr) == BITMOE_EHIP);
                    const size_t need = moe_expert_matmul_i8_workspace_bytes(E, R, N, K);
                    EXPECT(need % 256 == 0);
                    EXPECT(moe_expert_matmul_i8(&x, &w, ints, R, &y, ws, need, nullptr) == BITMOE_EHIP);
                    if (need)
                        EXPECT(moe_expert_matmul_i8(&x, &w, ints, R, &y, ws, need - 1, nullptr) == BITMOE_EWORKSPACE);
                }
    EXPECT(launches > 2000);
    for (int T : {0, 1, 2, 3, 100, 5000, 1 << 24})
        for (int H : {1, 7, 64, 512, 513, 1000, 2048, 2049, 4096, 4097, 7168, 8192, 8193, 16384}) {
            const bitmoe_rows m = rows(T, H), f = rows(T, H, BITMOE_F32), one = rows(1, H), of = rows(1, H, BITMOE_F32);
            const int rc = T ? BITMOE_EHIP : BITMOE_OK;
            EXPECT(moe_block_norm(&m, ws, &one, &f, 1.f, &f, ws, 1e-6f, &m, nullptr) == rc);
            EXPECT(moe_block_norm(nullptr, nullptr, nullptr, &m, 1.f, nullptr, ws, 1e-6f, &m, nullptr) == rc);
            const size_t need = moe_block_norm_backward_workspace_bytes(T, H);
            EXPECT(moe_block_norm_backward(&m, &f, &f, &m, ws, &one, 1.f, ws, 1e-6f, &m, &f, ws, &of, ws, BITMOE_F32, ws, need,
                                           nullptr) == BITMOE_EHIP);
            EXPECT(moe_block_norm_backward(&m, &m, &m, &m, ws, &m, 1.f, ws, 1e-6f, &m, &m, ws, T == 1 ? &one : &m, ws, BITMOE_BF16,
                                           ws, need, nullptr) == (BITMOE_EHIP));
            if (need)
                EXPECT(moe_block_norm_backward(&m, &f, &f, &m, ws, &one, 1.f, ws, 1e-6f, &m, &f, ws, &of, ws, BITMOE_F32, ws,
                                               need - 1, nullptr) == BITMOE_EWORKSPACE);
        }
    const bitmoe_rows x = rows(32, 100);
    for (int block : {0, 32, 64, 128}) {
        const bitmoe_rows8 q = rows8(32, 100, block);
        EXPECT(moe_quantize_rows(&x, &q, nullptr) == BITMOE_EHIP && moe_dequantize_rows(&q, &x, nullptr) == BITMOE_EHIP);
        EXPECT(moe_swiglu_rows8(&x, &x, &q, nullptr) == BITMOE_EHIP);
        const int rc = block ? BITMOE_EHIP : BITMOE_EINVAL;
        EXPECT(moe_swiglu_checkpoint(&x, &x, &x, &q, &q, nullptr) == rc);
        EXPECT(moe_swiglu_checkpoint_backward(&x, &q, &q, &x, &x, &x, nullptr) == rc);
    }
    std::printf(failures ? "rows8 sanitizer driver: %d check(s) failed\n" : "rows8 sanitizer driver: ok\n", failures);
    return failures ? 1 : 0;
}
