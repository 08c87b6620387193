// The matrix products for rows on 16-byte addresses.
//
// A stage is 32 of the contraction of a BM x BN tile, loaded from memory
// straight into LDS (global_load_lds, 16 bytes a lane, no registers) in a ring
// of four: when the matrix cores work on stage s, its operands are in
// registers already, those of s + 1 are being read from LDS, and s + 2 .. s + 4
// are on their way, so a load has three stages (3 x 1024 cycles at 256 x 256)
// to arrive.  One barrier a stage.
#pragma once

#include "gemm_util.h"

namespace bm {

constexpr int kTK = 32;             // contraction per stage
constexpr int kRing = 4;

// what a piece outside the operand reads
__device__ const uint4 kZeroPiece = {0, 0, 0, 0};

BM_DEV uint32_t lds_addr(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}
// 16 (4) bytes per lane to LDS, lane l's at `lds` (one for the wave) + 16 l
// (4 l).  In asm, because the compiler would wait for it before the next LDS
// read, of whatever stage; ring_barrier() waits instead.
BM_DEV void dma16(const void *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory");
}
BM_DEV void dma4(const void *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src) : "memory");
}
// all but this wave's last N loads have arrived, its LDS reads are done, and
// so for every wave of the workgroup
template <int N>
BM_DEV void ring_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// dynamic LDS of a tile: the ring; the output rows; for the weights' gradient
// each wave's ring of row maps (32 of A's, 32 of B's per stage).  The epilogue
// takes the ring's place.
template <int LAY, int BM, int BN, int WM, int WN>
struct TileLds {
    static constexpr int ring = kRing * (BM + BN) * kTK * 2;
    static constexpr int maps = ring + BM * 4;
    static constexpr int bytes = maps + (LAY == kGradWeights ? WM * WN * 4 * 64 * 4 : 0);
    static_assert(WM * WN * 32 * (BN / WN + 4) * 4 <= ring, "the epilogue's part");
    static_assert(bytes <= 160 * 1024, "");
};

template <int LAY, int DT, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN)
k_gemm_tile(GemmArgs g, int mtiles, int ntiles) {
    constexpr int NW = WM * WN, PA = BM * kTK / 8 / (64 * NW), PB = BN * kTK / 8 / (64 * NW);
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr bool AKC = LAY != kGradWeights, BKC = LAY == kForward;
    constexpr int kStage = (BM + BN) * kTK;        // elements
    constexpr int kLoads = PA + PB + (LAY == kGradWeights);
    static_assert(PA >= 1 && PB >= 1, "");
    extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
    Tile t;
    if (LAY == kGradWeights ? !find_tile_dw(g, mtiles, ntiles, blockIdx.x, &t)
                            : !find_tile<BM>(g, ntiles, blockIdx.x, &t))
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int m0 = t.m * BM, n0 = t.n * BN;
    const int kend = LAY == kGradWeights ? t.r1 - t.r0 : g.K;
    const int stages = (kend + kTK - 1) / kTK;
    const uint16_t *A = static_cast<const uint16_t *>(g.a.p);
    const uint16_t *B = static_cast<const uint16_t *>(g.b.p);
    if (LAY != kGradWeights) B += (int64_t)t.e * g.b_stride;
    const uint16_t *zero = reinterpret_cast<const uint16_t *>(&kZeroPiece);

    // Piece i of this thread in LDS order: tid + 64 NW i.  Its place in the
    // row does not depend on i (the rows of successive pieces differ by a
    // multiple of the swizzles' period), its row does.
    int ar, ac, br, bc;
    piece_at<AKC, BM, kTK>(tid, &ar, &ac);
    piece_at<BKC, BN, kTK>(tid, &br, &bc);
    constexpr int kRowA = AKC ? 16 * NW : 64 * NW * 8 / BM, kRowB = BKC ? 16 * NW : 64 * NW * 8 / BN;
    static_assert((kRowA % 16 == 0 || PA == 1) && (kRowB % 16 == 0 || PB == 1), "the swizzles' period");
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
            astep[i] = row >= 0 ? kTK : 0;
        }
    }
    if (BKC) {
#pragma unroll
        for (int i = 0; i < PB; i++) bp[i] = B + (int64_t)min(n0 + br + i * kRowB, g.N - 1) * g.b.ld + 8 * bc;
    }
    // KS: the column within the matrix
    const int acol = m0 + 8 * ac < g.M ? m0 + 8 * ac : 0, bcol = n0 + 8 * bc < g.N ? n0 + 8 * bc : 0;
    // the weights' gradient: the wave's own copy of the rows' maps, three stages
    // ahead of the loads that go by them
    int *maps = reinterpret_cast<int *>(reinterpret_cast<char *>(lds) + TileLds<LAY, BM, BN, WM, WN>::maps) + wave * 256;
    const uint32_t maps_at = lds_addr(maps);
    auto fetch_maps = [&](int s) {
        const int32_t *m = lane < 32 ? g.a.map : g.b.map;
        const int k = min(s * kTK + (lane & 31), kend - 1);
        dma4(m ? static_cast<const void *>(m + t.r0 + k) : zero, maps_at + (s & 3) * 256);
    };
    auto map_row = [&](const GemmRows &q, int at, int s, int k) {
        if (k >= kend) return -1;
        int m = t.r0 + k;
        if (q.map) {
            m = maps[(s & 3) * 64 + at];
            if (m < 0) return -1;
            m = divided(q, m);
        }
        return m < q.rows ? m : -1;
    };
    const uint32_t lds0 = lds_addr(lds) + wave * 1024;
    // load i of a stage (A's pieces, then B's, then the maps)
    auto load_one = [&](int s, int i) {
        const int k0 = s * kTK;
        const uint32_t la = lds0 + (s & 3) * (kStage * 2), lb = la + BM * kTK * 2;
        if (i < PA) {
            const uint16_t *p;
            if (AKC) {
                p = k0 + 8 * ac < kend ? ap[i] : zero;
                ap[i] += astep[i];
            } else {
                const int k = ar + i * kRowA, r = map_row(g.a, k, s, k0 + k);
                p = r >= 0 ? A + (int64_t)r * g.a.ld + acol : zero;
            }
            dma16(p, la + i * (NW * 1024));
        } else if (i < PA + PB) {
            const uint16_t *p;
            i -= PA;
            if (BKC) {
                p = k0 + 8 * bc < kend ? bp[i] : zero;
                bp[i] += kTK;
            } else {
                const int k = br + i * kRowB;
                const int r = LAY == kGradWeights ? map_row(g.b, 32 + k, s, k0 + k) : k0 + k < kend ? k0 + k : -1;
                p = r >= 0 ? B + (int64_t)r * g.b.ld + bcol : zero;
            }
            dma16(p, lb + i * (NW * 1024));
        } else {
            fetch_maps(s + 3);
        }
    };
    auto load = [&](int s) {
#pragma unroll
        for (int i = 0; i < kLoads; i++) load_one(s, i);
    };
    int *srow = reinterpret_cast<int *>(reinterpret_cast<char *>(lds) + TileLds<LAY, BM, BN, WM, WN>::ring);
    static_assert(BM <= 64 * NW, "");
    set_rows<LAY, BM>(g, t, m0, tid, srow);
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    s16x8 fa[2][TM], fb[2][TN];
    auto read_a = [&](int s, int i) {
        return frag<AKC, BM, kTK>(lds + (s & 3) * kStage, wm * (BM / WM) + 16 * i, 0, lane);
    };
    auto read_b = [&](int s, int j) {
        return frag<BKC, BN, kTK>(lds + (s & 3) * kStage + BM * kTK, wn * (BN / WN) + 16 * j, 0, lane);
    };
    // Stage s's products, in parts, each with its share of the reads of s + 1
    // before it and of the loads of s + 4 after it (into s's own place: its
    // operands are in registers).  Issued together after the barrier, the 32
    // loads of a stage hold up all that follows them: a CU takes about 16
    // cycles for each.
    auto step = [&](int s, s16x8 (&a)[TM], s16x8 (&b)[TN], s16x8 (&na)[TM], s16x8 (&nb)[TN]) {
        ring_barrier<2 * kLoads>();
        constexpr int kParts = TM >= 4 ? 4 : TM, kRows = TM / kParts;
#pragma unroll
        for (int c = 0; c < kParts; c++) {
#pragma unroll
            for (int j = c; j < TN; j += kParts) nb[j] = read_b(s + 1, j);
#pragma unroll
            for (int i = c * kRows; i < (c + 1) * kRows; i++) na[i] = read_a(s + 1, i);
            // (B first: a lane then holds four consecutive columns of one row)
#pragma unroll
            for (int i = c * kRows; i < (c + 1) * kRows; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j] = mfma16<DT>(b[j], a[i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = c; i < kLoads; i += kParts) load_one(s + 4, i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (stages > 0) {
        if (LAY == kGradWeights) {
            // (the maps of the stages that the first loads go by)
            for (int s = 0; s < 4; s++) fetch_maps(s);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            // load(s) fetches the maps of s + 3, load(0) of 3 again: the same values
        }
        for (int s = 0; s < 4; s++) load(s);
        ring_barrier<3 * kLoads>();
#pragma unroll
        for (int i = 0; i < TM; i++) fa[0][i] = read_a(0, i);
#pragma unroll
        for (int j = 0; j < TN; j++) fb[0][j] = read_b(0, j);
        for (int s = 0; s < stages; s += 2) {
            step(s, fa[0], fb[0], fa[1], fb[1]);
            if (s + 1 >= stages) break;
            step(s + 1, fa[1], fb[1], fa[0], fb[0]);
        }
    }
    // the epilogue writes where the ring's last loads go
    ring_barrier<0>();
    tile_epilogue<LAY, DT, TM, TN>(g, acc, reinterpret_cast<float *>(lds), srow + wm * (BM / WM), t.e,
                                   n0 + wn * (BN / WN), wave, lane);
}

}  // namespace bm
