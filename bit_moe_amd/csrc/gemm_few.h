// Forward products for groups of few rows (single tokens), bound by the
// weights: they go from memory straight into matrix-core operands.
//
// A workgroup makes NB = 16 / P outputs of up to RPP = NC * RP rows of a group
// (RP = 16 / P).  An operand's 16 rows are NB rows of W in P parts of the
// contraction, and the other's RP rows of x in the same P parts; of the 16 x 16
// product the P blocks on the diagonal are sums of one part each, added at the
// end.  P > 1 gives a small matrix more workgroups (512 outputs of one row: 128
// of 4 outputs each).  The 4 waves take a quarter of each part; lane l reads 8
// values at a time of its row, and the four lanes of a row 128 bytes in two
// loads (both operands order the contraction alike, in whatever order).
// Bound by the weights' bytes, the most a compute unit can have on their way:
// one row of 2048 x 7168 in 6.8 us (29 MB at 4.3 TB/s, about 2 us of it a
// launch; repeated, so out of the memory-side cache; 9.1 from HBM), of 16384 x 4096 in 22.1
// (134 MB at 6.1 TB/s).  x comes from L2 once per workgroup, at less than twice
// W's rate, which ends the kernel's use at about 16 rows.  Through LDS in the tiles' kernels the same row takes 11.3
// us: the parts' second launch and half-empty tiles.
#pragma once

#include "gemm_util.h"

namespace bm {

template <int DT, int P, int NC>
__global__ void __launch_bounds__(256)
k_gemm_few(GemmArgs g, int mtiles, int ntiles) {
    constexpr int NB = 16 / P, RP = 16 / P, RPP = NC * RP, U = NC == 1 ? 4 : 2;
    __shared__ float red[4][NC][16][17];
    Tile t;
    Tiles<kForward, RPP> list;
    list.init(g, mtiles, ntiles, blockIdx.x, gridDim.x);
    if (!list.next(g, &t)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, q = lane >> 4, in = i % NB, part = i / NB;
    const int r0 = t.r0 + t.m * RPP, n0 = t.n * NB;
    const int slice = ((g.K + 4 * P - 1) / (4 * P) + 63) / 64 * 64;
    const int kb = (part * 4 + wave) * slice + 16 * q;                 // this lane's first value
    const int kend = min((part * 4 + wave + 1) * slice, g.K);
    const uint16_t *w = static_cast<const uint16_t *>(g.b.p) + (int64_t)t.e * g.b_stride +
                        (int64_t)min(n0 + in, g.N - 1) * g.b.ld;
    const uint16_t *x[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int r = r0 + c * RP + in, row = r < t.r1 ? row_of(g.a, r) : -1;
        x[c] = row >= 0 ? static_cast<const uint16_t *>(g.a.p) + (int64_t)row * g.a.ld : nullptr;
    }
    auto read = [&](const uint16_t *p, int k) -> uint4 {
        if (!p || k >= kend) return make_uint4(0, 0, 0, 0);
        return k + 8 <= kend ? load16(p + k) : load16_part(p + k, kend - k);
    };
    struct Batch {
        uint4 w[2 * U], x[NC][2 * U];
    };
    // U steps of 64: where every lane's values are there, its loads are issued
    // together
    auto load = [&](int b, Batch &o) __attribute__((always_inline)) {
        const int k = kb + b * (64 * U);
        if (__all(k + 64 * (U - 1) + 16 <= kend)) {
#pragma unroll
            for (int u = 0; u < 2 * U; u++) o.w[u] = load16(w + k + (u >> 1) * 64 + (u & 1) * 8);
#pragma unroll
            for (int c = 0; c < NC; c++) {
                if (x[c]) {
#pragma unroll
                    for (int u = 0; u < 2 * U; u++) o.x[c][u] = load16(x[c] + k + (u >> 1) * 64 + (u & 1) * 8);
                } else {
#pragma unroll
                    for (int u = 0; u < 2 * U; u++) o.x[c][u] = make_uint4(0, 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < 2 * U; u++) {
                o.w[u] = read(w, k + (u >> 1) * 64 + (u & 1) * 8);
#pragma unroll
                for (int c = 0; c < NC; c++) o.x[c][u] = read(x[c], k + (u >> 1) * 64 + (u & 1) * 8);
            }
        }
    };
    f32x4 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Batch &o) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 2 * U; u++)
#pragma unroll
            for (int c = 0; c < NC; c++)
                acc[c] = mfma16<DT>(__builtin_bit_cast(s16x8, o.w[u]), __builtin_bit_cast(s16x8, o.x[c][u]), acc[c]);
    };
    const int batches = (slice + 64 * U - 1) / (64 * U);
    Batch a, b;
    load(0, a);
    for (int j = 0; j < batches; j += 2) {
        if (j + 1 < batches) load(j + 1, b);
        multiply(a);
        if (j + 1 >= batches) break;
        if (j + 2 < batches) load(j + 2, a);
        multiply(b);
    }
    // lane l holds outputs 4 (l / 16) + 0..3 of the row l % 16
#pragma unroll
    for (int c = 0; c < NC; c++)
#pragma unroll
        for (int j = 0; j < 4; j++) red[wave][c][4 * q + j][i] = acc[c][j];
    __syncthreads();
    for (int o = tid; o < RPP * NB; o += 256) {
        const int n = o % NB, r = o / NB % RP, c = o / (NB * RP);
        if (r0 + c * RP + r >= t.r1 || n0 + n >= g.N) continue;
        const int row = row_of(g.c, r0 + c * RP + r);
        if (row < 0) continue;
        float v[1] = {0.f}, bias[1] = {0.f}, res[1] = {0.f};
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
            for (int s = 0; s < 4; s++) v[0] += red[s][c][p * NB + n][p * NB + r];
        if (g.bias) load_row<DT>(g.bias, n0 + n, false, bias);
        if (g.res) load_row<DT>(g.res, (int64_t)row * g.ld_res + n0 + n, g.res_f32, res);
        finish<kForward, DT>(g, t.e, 0, row, n0 + n, v, bias, res);
    }
}

}  // namespace bm
