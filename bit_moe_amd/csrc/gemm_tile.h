// The matrix products for rows on 16-byte addresses: tiles that go from
// memory straight into LDS (global_load_lds, 16 bytes a lane) while the stage
// before is multiplied.
#pragma once

#include "gemm_util.h"

namespace bm {

// what a piece outside the operand reads
__device__ const uint4 kZeroPiece = {0, 0, 0, 0};

BM_DEV uint32_t lds_addr(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}
// 16 bytes per lane to LDS, lane l's at `lds` (one for the wave) + 16 l.  In
// asm, because the compiler would wait for it before the next LDS read of
// another stage; tile_barrier() waits instead.
BM_DEV void dma16(const void *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory");
}
// every wave's loads have arrived and its LDS reads are done
BM_DEV void tile_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int LAY, int DT, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN)
k_gemm_tile(GemmArgs g, int mtiles, int ntiles) {
    constexpr int NW = WM * WN, PA = BM * kBK / 8 / (64 * NW), PB = BN * kBK / 8 / (64 * NW);
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr bool AKC = LAY != kGradWeights, BKC = LAY == kForward;
    constexpr int kStage = (BM + BN) * kBK;        // elements
    extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
    Tile t;
    if (LAY == kGradWeights ? !find_tile_dw(g, mtiles, ntiles, blockIdx.x, &t)
                            : !find_tile<BM>(g, ntiles, blockIdx.x, &t))
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int m0 = t.m * BM, n0 = t.n * BN;
    const int kend = LAY == kGradWeights ? t.r1 - t.r0 : g.K;
    const uint16_t *A = static_cast<const uint16_t *>(g.a.p);
    const uint16_t *B = static_cast<const uint16_t *>(g.b.p);
    if (LAY != kGradWeights) B += (int64_t)t.e * g.b_stride;
    const uint16_t *zero = reinterpret_cast<const uint16_t *>(&kZeroPiece);

    // Piece i of this thread in LDS order: tid + 64 NW i.  Its place in the
    // row does not depend on i (the rows of successive pieces differ by a
    // multiple of the swizzles' period), its row does.
    int ar, ac, br, bc;
    piece_at<AKC, BM>(tid, &ar, &ac);
    piece_at<BKC, BN>(tid, &br, &bc);
    constexpr int kRowA = AKC ? 8 * NW : 64 * NW * 8 / BM, kRowB = BKC ? 8 * NW : 64 * NW * 8 / BN;
    static_assert(kRowA % 16 == 0 && kRowB % 16 == 0, "the swizzles' period");
    // KC: each piece's address, and how far it moves per stage (0: the zero
    // piece).  Rows past the group, and columns past the matrix, read its
    // last row (their results are not stored).
    const uint16_t *ap[PA], *bp[PB];
    int astep[PA];
    if (AKC) {
#pragma unroll
        for (int i = 0; i < PA; i++) {
            const int row = row_of(g.a, min(t.r0 + m0 + ar + i * kRowA, t.r1 - 1));
            ap[i] = row >= 0 ? A + (int64_t)row * g.a.ld + 8 * ac : zero;
            astep[i] = row >= 0 ? kBK : 0;
        }
    }
    if (BKC) {
#pragma unroll
        for (int i = 0; i < PB; i++) bp[i] = B + (int64_t)min(n0 + br + i * kRowB, g.N - 1) * g.b.ld + 8 * bc;
    }
    // KS: the column within the matrix, and the rows one stage ahead, as the
    // map gives them (what is made of them waits for the next stage's loads,
    // or the map's own would be waited for here)
    const int acol = m0 + 8 * ac < g.M ? m0 + 8 * ac : 0, bcol = n0 + 8 * bc < g.N ? n0 + 8 * bc : 0;
    int arow[PA], brow[PB];
    auto fetch = [&](const GemmRows &q, int k) { return k >= kend ? -1 : q.map ? q.map[t.r0 + k] : t.r0 + k; };
    auto row_at = [&](const GemmRows &q, int m) {
        if (m < 0) return -1;
        if (q.map) m = divided(q, m);
        return m < q.rows ? m : -1;
    };
    auto fetch_rows = [&](int k0) {
        if (LAY == kGradWeights) {
#pragma unroll
            for (int i = 0; i < PA; i++) arow[i] = fetch(g.a, k0 + ar + i * kRowA);
#pragma unroll
            for (int i = 0; i < PB; i++) brow[i] = fetch(g.b, k0 + br + i * kRowB);
        }
    };
    const uint32_t lds0 = lds_addr(lds) + wave * 1024;
    auto load = [&](int k0, int buf) {
        const uint32_t la = lds0 + buf * (kStage * 2), lb = la + BM * kBK * 2;
#pragma unroll
        for (int i = 0; i < PA; i++) {
            const uint16_t *p;
            if (AKC) {
                p = k0 + 8 * ac < kend ? ap[i] : zero;
                ap[i] += astep[i];
            } else {
                const int r = row_at(g.a, arow[i]);
                p = r >= 0 ? A + (int64_t)r * g.a.ld + acol : zero;
            }
            dma16(p, la + i * (NW * 1024));
        }
#pragma unroll
        for (int i = 0; i < PB; i++) {
            const uint16_t *p;
            if (BKC) {
                p = k0 + 8 * bc < kend ? bp[i] : zero;
                bp[i] += kBK;
            } else {
                const int k = k0 + br + i * kRowB, r = LAY == kGradWeights ? row_at(g.b, brow[i]) : k < kend ? k : -1;
                p = r >= 0 ? B + (int64_t)r * g.b.ld + bcol : zero;
            }
            dma16(p, lb + i * (NW * 1024));
        }
        fetch_rows(k0 + kBK);
    };
    int *srow = reinterpret_cast<int *>(lds + 2 * kStage);
    static_assert(BM <= 64 * NW && NW * 32 * (BN / WN + 4) * 4 <= 4 * kStage, "");
    set_rows<LAY, BM>(g, t, m0, tid, srow);
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    fetch_rows(0);
    if (kend > 0) load(0, 0);
    int buf = 0;
    for (int k0 = 0; k0 < kend; k0 += kBK, buf ^= 1) {
        tile_barrier();
        if (k0 + kBK < kend) load(k0 + kBK, buf ^ 1);
        const uint16_t *sa = lds + buf * kStage, *sb = sa + BM * kBK;
#pragma unroll
        for (int kk = 0; kk < kBK; kk += 32) {
            s16x8 fa[TM], fb[TN];
#pragma unroll
            for (int j = 0; j < TN; j++) fb[j] = frag<BKC, BN>(sb, wn * (BN / WN) + 16 * j, kk, lane);
#pragma unroll
            for (int i = 0; i < TM; i++) fa[i] = frag<AKC, BM>(sa, wm * (BM / WM) + 16 * i, kk, lane);
            // (B first: a lane then holds four consecutive columns of one row)
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j] = mfma16<DT>(fb[j], fa[i], acc[i][j]);
        }
    }
    tile_barrier();
    tile_epilogue<LAY, DT, TM, TN>(g, acc, reinterpret_cast<float *>(lds), srow + wm * (BM / WM), t.e,
                                   n0 + wn * (BN / WN), wave, lane);
}

}  // namespace bm
