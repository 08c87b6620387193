// Matrix products of the 16-bit expert layer: forward, rows' gradient and
// weights' gradient over groups of rows of any size, C = A B^T on
// v_mfma_f32_16x16x32 with fp32 accumulation.
//
// k_gemm: rows of any alignment.  A workgroup of 4 waves makes a 128 x 128
// tile (64 x 64 a wave); a stage of 64 of the contraction is loaded into
// registers while the one before it is multiplied out of LDS.
#include "gemm_util.h"

namespace {

using namespace bm;

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
    __shared__ __attribute__((aligned(16))) uint16_t sa[BM * kBK];
    __shared__ __attribute__((aligned(16))) uint16_t sb[BN * kBK];
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
    const int mend = LAY == kGradWeights ? g.M : t.r1 - t.r0;
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const int m = m0 + wm * (BM / WM) + 16 * i + (lane & 15);
        if (m >= mend) continue;
#pragma unroll
        for (int j = 0; j < TN; j++) {
            float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            finish4<LAY>(g, t.e, LAY == kGradWeights ? m : t.r0 + m, n0 + wn * (BN / WN) + 16 * j + 4 * (lane >> 4), v);
        }
    }
}

template <int LAY, int DT>
int launch_one(const GemmArgs &g, hipStream_t s) {
    constexpr int BM = 128, BN = 128;
    const int64_t nt = (g.N + BN - 1) / BN;
    int64_t mt, items;
    if (LAY == kGradWeights) {
        mt = (g.M + BM - 1) / BM;
        items = g.E * mt * nt;
    } else {
        // row tiles of all groups, at most
        mt = g.R / BM + (g.E < g.R ? g.E : g.R);
        items = mt * nt;
    }
    const int64_t grid = (items + 7) / 8 * 8;
    if (grid * 256 >= (int64_t)1 << 32) return BITMOE_EUNSUPPORTED;
    k_gemm<LAY, DT, BM, BN, 2, 2><<<(int)grid, 256, 0, s>>>(g, (int)mt, (int)nt);
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
