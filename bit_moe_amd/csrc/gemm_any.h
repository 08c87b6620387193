// The matrix products for rows of any alignment: a workgroup of 4 waves makes a
// 128 x 128 tile (64 x 64 a wave); a stage of 64 of the contraction is loaded
// into registers while the one before it is multiplied out of LDS.  Bound by
// that way through the registers, 8 loads a thread and stage at addresses
// tested one by one, and its LDS writes: 8192 x 2048 x 7168 one element off
// 16 bytes in 358 us forward (672 TFLOP/s), 380 as rows' gradient and 575 as
// weights' gradient, 1.8, 1.75 and 2.9 times those of rows on 16-byte addresses;
// where the widths are odd too (2049 x 7167) 453, 474 and 1314.
#pragma once

#include "gemm_util.h"

namespace bm {

// 8 elements of a row of the operand (nullptr: zeros) from c8, up to `end`
BM_DEV uint4 load_piece(const uint16_t *row, int c8, int end) {
    if (!row || c8 >= end) return make_uint4(0, 0, 0, 0);
    if (c8 + 8 <= end) return load16(row + c8);
    return load16_part(row + c8, end - c8);
}

// PARTS (gradients): A is in two parts (g.a_low); the low one first, its sums
// scaled before the high one's.  (An instance of its own: in one for both the
// weights' gradient took 260 registers, which is one workgroup a unit, not two.)
template <int LAY, int DT, int BM, int BN, int WM, int WN, bool PARTS>
__global__ void __launch_bounds__(64 * WM * WN)
k_gemm(GemmArgs g, int mtiles, int ntiles) {
    constexpr int NT = 64 * WM * WN, PA = BM * kBK / 8 / NT, PB = BN * kBK / 8 / NT;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr bool AKC = LAY != kGradWeights, BKC = LAY == kForward;
    // the stage, and after it the epilogue's part
    __shared__ __attribute__((aligned(16))) uint16_t lds[(BM + BN) * kBK];
    static_assert(sizeof(lds) >= WM * WN * epilogue_floats<TN>() * 4, "");
    __shared__ int srow[BM];
    uint16_t *sa = lds, *sb = lds + BM * kBK;
    Tile t;
    Tiles<LAY, BM> list;
    list.init(g, mtiles, ntiles * g.splits, blockIdx.x, gridDim.x);
    if (!list.next(g, &t) || t.m < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const Span k = span_of<LAY>(g, &t, ntiles);
    const int m0 = t.m * BM, n0 = t.n * BN;
    const int kend = k.end;
    const uint16_t *A = static_cast<const uint16_t *>(g.a.p);
    const uint16_t *B = static_cast<const uint16_t *>(g.b.p);
    if (LAY != kGradWeights) B += (int64_t)t.e * g.b_stride;
    if (PARTS) A += g.a_low;

    // pieces along a row keep their row over the stages
    const uint16_t *arow[PA], *brow[PB];
    int ar[PA], ac[PA], br[PB], bc[PB];
#pragma unroll
    for (int i = 0; i < PA; i++) {
        piece_at<AKC, BM>(tid + i * NT, &ar[i], &ac[i]);
        arow[i] = nullptr;
        if (AKC) {
            const int r = t.r0 + m0 + ar[i];
            const int row = r < t.r1 ? row_of(g.a, r) : -1;
            if (row >= 0) arow[i] = A + (int64_t)row * g.a.ld;
        }
    }
#pragma unroll
    for (int i = 0; i < PB; i++) {
        piece_at<BKC, BN>(tid + i * NT, &br[i], &bc[i]);
        brow[i] = nullptr;
        if (BKC && n0 + br[i] < g.N) brow[i] = B + (int64_t)(n0 + br[i]) * g.b.ld;
    }
    uint4 va[PA], vb[PB];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < PA; i++) {
            if (AKC) {
                va[i] = load_piece(arow[i], k0 + 8 * ac[i], kend);
            } else {
                // (a row that either operand lacks adds nothing, whatever the other holds)
                const int kr = k0 + ar[i];
                const int row = kr < kend && row_of(g.b, t.r0 + kr) >= 0 ? row_of(g.a, t.r0 + kr) : -1;
                va[i] = load_piece(row >= 0 ? A + (int64_t)row * g.a.ld : nullptr, m0 + 8 * ac[i], g.M);
            }
        }
#pragma unroll
        for (int i = 0; i < PB; i++) {
            if (BKC) {
                vb[i] = load_piece(brow[i], k0 + 8 * bc[i], kend);
            } else if (LAY == kGradRows) {
                const int kr = k0 + br[i];
                vb[i] = load_piece(kr < kend ? B + (int64_t)kr * g.b.ld : nullptr, n0 + 8 * bc[i], g.N);
            } else {
                const int kr = k0 + br[i];
                const int row = kr < kend && row_of(g.a, t.r0 + kr) >= 0 ? row_of(g.b, t.r0 + kr) : -1;
                vb[i] = load_piece(row >= 0 ? B + (int64_t)row * g.b.ld : nullptr, n0 + 8 * bc[i], g.N);
            }
        }
    };
    set_rows<LAY, BM>(g, t, m0, tid, srow);
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (bool low = PARTS;; low = false) {
        if (k.beg < kend) load(k.beg);
        for (int k0 = k.beg; k0 < kend; k0 += kBK) {
#pragma unroll
            for (int i = 0; i < PA; i++) *reinterpret_cast<uint4 *>(sa + (tid + i * NT) * 8) = va[i];
#pragma unroll
            for (int i = 0; i < PB; i++) *reinterpret_cast<uint4 *>(sb + (tid + i * NT) * 8) = vb[i];
            __syncthreads();
            if (k0 + kBK < kend) load(k0 + kBK);
#pragma unroll
            for (int kk = 0; kk < kBK; kk += 32) {
                s16x8 fa[TM], fb[TN];
#pragma unroll
                for (int i = 0; i < TM; i++) fa[i] = frag<AKC, BM>(sa, wm * (BM / WM) + 16 * i, kk, lane);
#pragma unroll
                for (int j = 0; j < TN; j++) fb[j] = frag<BKC, BN>(sb, wn * (BN / WN) + 16 * j, kk, lane);
                // (B first: a lane then holds four consecutive columns of one row)
#pragma unroll
                for (int i = 0; i < TM; i++)
#pragma unroll
                    for (int j = 0; j < TN; j++) acc[i][j] = mfma16<DT>(fb[j], fa[i], acc[i][j]);
            }
            __syncthreads();
        }
        if (!PARTS) break;
        const float scale = low ? 1.f / low_scale<DT>() : 2.f;
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++) acc[i][j] *= scale;
        if (!low) break;
        A -= g.a_low;
#pragma unroll
        for (int i = 0; i < PA; i++)
            if (arow[i]) arow[i] -= g.a_low;
    }
    __syncthreads();         // (srow, where the loop did not run)
    tile_epilogue<LAY, DT, BM, BN, 1>(g, acc, reinterpret_cast<float *>(lds), srow, t.e, k.split, n0, wm * (BM / WM),
                                      wn * (BN / WN), wave, lane);
}

}  // namespace bm
