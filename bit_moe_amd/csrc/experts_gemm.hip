// Matrix products of the 16-bit expert layer: forward, rows' gradient and
// weights' gradient over groups of rows of any size, C = A B^T on
// v_mfma_f32_16x16x32 with fp32 accumulation.
//
// k_gemm: rows of any alignment.  A workgroup of 4 waves makes a 128 x 128
// tile (64 x 64 a wave); a stage of 64 of the contraction is loaded into
// registers while the one before it is multiplied out of LDS.
#include <algorithm>

#include "gemm_tile.h"

namespace {

using namespace bm;
using bm_host::cu_count;


// 8 elements of an operand's stage: row `row` of the rows it runs along
// (KC: an output row, KS: a step of the contraction), elements c8.. of it
struct Piece {
    const uint16_t *p;      // the row's first element; nullptr: zeros
    int c8;
};

BM_DEV uint4 load_piece(const uint16_t *row, int c8, int end) {
    if (!row || c8 >= end) return make_uint4(0, 0, 0, 0);
    if (c8 + 8 <= end) return load16(row + c8);
    return load16_part(row + c8, end - c8);
}

template <int LAY, int DT, int BM, int BN, int WM, int WN>
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
    list.init(g, mtiles, ntiles, blockIdx.x, gridDim.x);
    if (!list.next(g, &t) || t.m < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int m0 = t.m * BM, n0 = t.n * BN;
    const int kend = LAY == kGradWeights ? t.r1 - t.r0 : g.K;
    const uint16_t *A = static_cast<const uint16_t *>(g.a.p);
    const uint16_t *B = static_cast<const uint16_t *>(g.b.p);
    if (LAY != kGradWeights) B += (int64_t)t.e * g.b_stride;

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
                const int k = k0 + ar[i], row = k < kend ? row_of(g.a, t.r0 + k) : -1;
                va[i] = load_piece(row >= 0 ? A + (int64_t)row * g.a.ld : nullptr, m0 + 8 * ac[i], g.M);
            }
        }
#pragma unroll
        for (int i = 0; i < PB; i++) {
            if (BKC) {
                vb[i] = load_piece(brow[i], k0 + 8 * bc[i], kend);
            } else if (LAY == kGradRows) {
                const int k = k0 + br[i];
                vb[i] = load_piece(k < kend ? B + (int64_t)k * g.b.ld : nullptr, n0 + 8 * bc[i], g.N);
            } else {
                const int k = k0 + br[i], row = k < kend ? row_of(g.b, t.r0 + k) : -1;
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
    if (kend > 0) load(0);
    for (int k0 = 0; k0 < kend; k0 += kBK) {
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
    __syncthreads();         // (srow, where the loop did not run)
    tile_epilogue<LAY, DT, BM, BN, 1>(g, acc, reinterpret_cast<float *>(lds), srow, t.e, n0, wm * (BM / WM),
                                      wn * (BN / WN), wave, lane);
}

// rows that all begin on 16-byte addresses, whole 8-element pieces
bool on16(const void *p, int64_t ld, int cols) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && cols % 8 == 0;
}
template <int LAY>
bool pieces_whole(const GemmArgs &g) {
    if (LAY == kGradWeights) return on16(g.a.p, g.a.ld, g.M) && on16(g.b.p, g.b.ld, g.N);
    return on16(g.a.p, g.a.ld, g.K) && on16(g.b.p, g.b.ld, LAY == kForward ? g.K : g.N) &&
           (g.E == 1 || g.b_stride % 8 == 0);
}

template <int LAY, int BM, int BN>
int64_t tiles(const GemmArgs &g, int *mt, int *nt) {
    *nt = (g.N + BN - 1) / BN;
    // (rows: the tiles of all groups, at most)
    *mt = LAY == kGradWeights ? (g.M + BM - 1) / BM : g.R / BM + (g.E < g.R ? g.E : g.R);
    if (LAY == kGradWeights) return (int64_t)g.E * dw_eighth(*mt, *nt) * 8;
    return ((int64_t)*mt * *nt + 7) / 8 * 8;
}

template <int LAY, int DT, int BM, int BN, int WM, int WN>
int launch_tile(const GemmArgs &g, hipStream_t s) {
    int mt, nt;
    const int64_t grid = tiles<LAY, BM, BN>(g, &mt, &nt);
    constexpr int lds = TileLds<LAY, BM, BN, WM, WN>::bytes;
    // as many workgroups as fit the GPU together, each for several tiles
    const int64_t most = (int64_t)cu_count() * (160 * 1024 / lds);
    // (LDS above 64 KiB must be opted into per kernel and device)
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(k_gemm_tile<LAY, DT, BM, BN, WM, WN>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    k_gemm_tile<LAY, DT, BM, BN, WM, WN><<<(int)std::min(grid, std::max<int64_t>(most / 8 * 8, 8)), 64 * WM * WN, lds, s>>>(g, mt, nt);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

template <int LAY, int DT>
int launch_one(const GemmArgs &g, hipStream_t s) {
    if (pieces_whole<LAY>(g)) return launch_tile<LAY, DT, 256, 256, 2, 4>(g, s);
    int mt, nt;
    const int64_t grid = tiles<LAY, 128, 128>(g, &mt, &nt);
    if (grid * 256 >= (int64_t)1 << 32) return BITMOE_EUNSUPPORTED;
    k_gemm<LAY, DT, 128, 128, 2, 2><<<(int)grid, 256, 0, s>>>(g, mt, nt);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

}  // namespace

namespace bm_host {

size_t gemm_ws_bytes(int, const GemmArgs &) { return 0; }

int launch_gemm(int layout, int dtype, const GemmArgs &g, void *, hipStream_t s) {
    switch (layout * 2 + (dtype == BITMOE_F16)) {
        case 0: return launch_one<kForward, BITMOE_BF16>(g, s);
        case 1: return launch_one<kForward, BITMOE_F16>(g, s);
        case 2: return launch_one<kGradRows, BITMOE_BF16>(g, s);
        case 3: return launch_one<kGradRows, BITMOE_F16>(g, s);
        case 4: return launch_one<kGradWeights, BITMOE_BF16>(g, s);
        case 5: return launch_one<kGradWeights, BITMOE_F16>(g, s);
    }
    return BITMOE_EINVAL;
}

}  // namespace bm_host
