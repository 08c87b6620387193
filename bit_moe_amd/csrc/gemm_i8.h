// Products in 8 bits: their epilogue, and the kernels for codes of any alignment and
// for few rows.  8192^3 391 to 422 us in the tile kernel from run to run (2.8 to 2.6 POPS),
// 8192 x 4096 x 7168 184 to 192 (2.6 to 2.5), 256 groups of 64 rows at 5.5 TB/s.
#pragma once

#include "gemm_util.h"

namespace bm {

// the scale of expert e's output n (of the last one, past it), and of the call's row
// r (0 for one that the map does not give)
BM_DEV float col_scale(const GemmArgs &g, int e, int n) { return g.b_scale[e * g.b_scale_stride + min(n, g.N - 1)]; }
BM_DEV float row_scale(const GemmArgs &g, int r) {
    const int row = row_of(g.a, r);
    return row >= 0 ? g.a_scale[row * g.a_ld_scale] : 0.f;
}

// The waves' int32 sums to memory, as tile_epilogue does it: a lane's 4 columns
// of a row become 8 through LDS.  A value is (sum * row's scale) * column's
// scale in fp32, rounded once to its type; the sum to fp32 is one rounding more
// (from 2^24).  srow, sscale, scol: output row (or -1) and scale of each of the tile's
// rows, scale of each of its columns (in LDS: a load here would wait for those of the
// next tile, which are on their way).
template <int DT, int BM, int BN, int HALVES, int TM, int TN>
BM_DEV void i8_epilogue(const GemmArgs &g, const i32x4 (&acc)[TM][TN], float *lds, const int *srow, const float *sscale,
                        const float *scol, int split, int n0, int m_at, int n_at, int wave, int lane) {
    constexpr int MR = 16 * TM / HALVES, TH = TN / 2, CW = 16 * TH;      // columns at a time
    constexpr int LDW = CW + 4, LPR = CW / 8, RPI = 64 / LPR, IT = 16 / RPI;
    int *sw = reinterpret_cast<int *>(lds) + wave * epilogue_floats<TN>();
    const int r0 = lane / LPR, c = (lane % LPR) * 8;
    const int nn[2] = {n0 + n_at + c, n0 + n_at + c + (HALVES == 2 ? BN / 2 : CW)};
    float cs[2][8];
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int j = 0; j < 8; j++)
            cs[h][j] = scol[nn[h] - n0 + j];
#pragma unroll
    for (int q = 0; q < TM; q++) {
        int rows[IT];
        float rs[IT];
#pragma unroll
        for (int it = 0; it < IT; it++) {
            const int m = 16 * q + it * RPI + r0, at = m / MR * (BM / 2) + m_at + m % MR;
            rows[it] = srow[at];
            rs[it] = sscale[at];
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int j = 0; j < TH; j++)
                *reinterpret_cast<i32x4 *>(sw + (lane & 15) * LDW + 16 * j + 4 * (lane >> 4)) = acc[q][h * TH + j];
            wave_together();
#pragma unroll
            for (int it = 0; it < IT; it++) {
                const int r = it * RPI + r0;
                const i32x4 a = *reinterpret_cast<const i32x4 *>(sw + r * LDW + c);
                const i32x4 b = *reinterpret_cast<const i32x4 *>(sw + r * LDW + c + 4);
                const int left = g.N - nn[h];
                if (rows[it] < 0 || left <= 0) continue;
                const int sum[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                float v[8];
                const int64_t at = split * g.c_split + (int64_t)rows[it] * g.c.ld + nn[h];
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] = g.raw ? __int_as_float(sum[j]) : (float)sum[j] * rs[it] * cs[h][j];
                store8<DT - kI8>(const_cast<void *>(g.c.p), at, min(left, 8), g.c_f32, v);
            }
            wave_together();
        }
    }
}

struct __attribute__((packed, aligned(1))) C128 { uint32_t w[4]; };
BM_DEV uint4 code_piece(const uint8_t *p) {
    const C128 u = *reinterpret_cast<const C128 *>(p);
    return make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
}
// 16 codes of a row (nullptr: zeros) from k, up to `end`
BM_DEV uint4 load_codes(const uint8_t *row, int k, int end) {
    if (!row || k >= end) return make_uint4(0, 0, 0, 0);
    if (k + 16 <= end) return code_piece(row + k);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; j++)
        if (k + j < end) w[j >> 2] |= (uint32_t)row[k + j] << (8 * (j & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of any alignment: a workgroup of 4 waves makes a 128 x 128 tile (64 x 64
// a wave); a stage of 128 codes is loaded into registers while the one before it
// is multiplied out of LDS (the layout is the 16-bit products': a code pair is an
// element there).
template <int DT>
__global__ void __launch_bounds__(256)
k_i8_any(GemmArgs g, int mtiles, int ntiles) {
    constexpr int BM = 128, BN = 128, P = 4, TM = 4, TN = 4, STAGE = 2 * kBK;
    __shared__ __attribute__((aligned(16))) uint16_t lds[(BM + BN) * kBK];
    static_assert(sizeof(lds) >= 4 * epilogue_floats<TN>() * 4, "");
    __shared__ int srow[BM];
    __shared__ float sscale[BM], scol[BN];
    uint16_t *sa = lds, *sb = lds + BM * kBK;
    Tile t;
    Tiles<kForward, BM> list;
    list.init(g, mtiles, ntiles * g.splits, blockIdx.x, gridDim.x);
    if (!list.next(g, &t)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const Span k = span_of<kForward>(g, &t, ntiles);
    const int m0 = t.m * BM, n0 = t.n * BN;
    const uint8_t *A = static_cast<const uint8_t *>(g.a.p);
    const uint8_t *B = static_cast<const uint8_t *>(g.b.p) + (int64_t)t.e * g.b_stride;
    const uint8_t *arow[P], *brow[P];
    int col[P];
#pragma unroll
    for (int i = 0; i < P; i++) {
        int r;
        piece_at<true, BM>(tid + i * 256, &r, &col[i]);
        const int row = t.r0 + m0 + r < t.r1 ? row_of(g.a, t.r0 + m0 + r) : -1;
        arow[i] = row >= 0 ? A + (int64_t)row * g.a.ld : nullptr;
        brow[i] = n0 + r < g.N ? B + (int64_t)(n0 + r) * g.b.ld : nullptr;
    }
    uint4 va[P], vb[P];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < P; i++) va[i] = load_codes(arow[i], k0 + 16 * col[i], k.end);
#pragma unroll
        for (int i = 0; i < P; i++) vb[i] = load_codes(brow[i], k0 + 16 * col[i], k.end);
    };
    set_rows<kForward, BM>(g, t, m0, tid, srow);
    if (tid < BM) sscale[tid] = !g.raw && m0 + tid < t.r1 - t.r0 ? row_scale(g, t.r0 + m0 + tid) : 0.f;
    if (tid < BN) scol[tid] = g.raw ? 0.f : col_scale(g, t.e, n0 + tid);
    i32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = i32x4{0, 0, 0, 0};
    if (k.beg < k.end) load(k.beg);
    for (int k0 = k.beg; k0 < k.end; k0 += STAGE) {
#pragma unroll
        for (int i = 0; i < P; i++) *reinterpret_cast<uint4 *>(sa + (tid + i * 256) * 8) = va[i];
#pragma unroll
        for (int i = 0; i < P; i++) *reinterpret_cast<uint4 *>(sb + (tid + i * 256) * 8) = vb[i];
        __syncthreads();
        if (k0 + STAGE < k.end) load(k0 + STAGE);
#pragma unroll
        for (int kk = 0; kk < kBK; kk += 32) {
            s16x8 fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; i++) fa[i] = frag<true, BM>(sa, wm * 64 + 16 * i, kk, lane);
#pragma unroll
            for (int j = 0; j < TN; j++) fb[j] = frag<true, BN>(sb, wn * 64 + 16 * j, kk, lane);
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j] = mfma16<DT>(fb[j], fa[i], acc[i][j]);
        }
        __syncthreads();
    }
    __syncthreads();         // (srow, where the loop did not run)
    i8_epilogue<DT, BM, BN, 1>(g, acc, reinterpret_cast<float *>(lds), srow, sscale, scol, k.split, n0, wm * 64, wn * 64,
                               wave, lane);
}

// Few rows (single tokens), as k_gemm_few: the weights go from memory straight
// into matrix-core operands.  A workgroup makes NB = 16 / P outputs of up to RPP =
// NC * RP rows of a group; P > 1 parts of the contraction lie side by side in an
// operand's 16 rows, whose diagonal blocks of the product are added at the end
// with the four waves' (in int32: exact, in any order).
template <int DT, int P, int NC>
__global__ void __launch_bounds__(256)
k_i8_few(GemmArgs g, int mtiles, int ntiles) {
    constexpr int NB = 16 / P, RP = 16 / P, RPP = NC * RP, U = NC == 1 ? 4 : 2;
    __shared__ int red[4][NC][16][17];
    Tile t;
    Tiles<kForward, RPP> list;
    list.init(g, mtiles, ntiles, blockIdx.x, gridDim.x);
    if (!list.next(g, &t)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, q = lane >> 4, in = i % NB, part = i / NB;
    const int r0 = t.r0 + t.m * RPP, n0 = t.n * NB;
    const int slice = ((g.K + 4 * P - 1) / (4 * P) + 127) / 128 * 128;
    const int kb = (part * 4 + wave) * slice + 32 * q;                 // this lane's first code
    const int kend = min((part * 4 + wave + 1) * slice, g.K);
    const uint8_t *w = static_cast<const uint8_t *>(g.b.p) + (int64_t)t.e * g.b_stride +
                       (int64_t)min(n0 + in, g.N - 1) * g.b.ld;
    const uint8_t *x[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int r = r0 + c * RP + in, row = r < t.r1 ? row_of(g.a, r) : -1;
        x[c] = row >= 0 ? static_cast<const uint8_t *>(g.a.p) + (int64_t)row * g.a.ld : nullptr;
    }
    struct Batch {
        uint4 w[2 * U], x[NC][2 * U];
    };
    // U steps of 128: where every lane's codes are there, its loads are issued
    // together
    auto load = [&](int b, Batch &o) __attribute__((always_inline)) {
        const int k = kb + b * (128 * U);
        if (__all(k + 128 * (U - 1) + 32 <= kend)) {
#pragma unroll
            for (int u = 0; u < 2 * U; u++) o.w[u] = code_piece(w + k + (u >> 1) * 128 + (u & 1) * 16);
#pragma unroll
            for (int c = 0; c < NC; c++) {
                if (x[c]) {
#pragma unroll
                    for (int u = 0; u < 2 * U; u++) o.x[c][u] = code_piece(x[c] + k + (u >> 1) * 128 + (u & 1) * 16);
                } else {
#pragma unroll
                    for (int u = 0; u < 2 * U; u++) o.x[c][u] = make_uint4(0, 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < 2 * U; u++) {
                const int at = k + (u >> 1) * 128 + (u & 1) * 16;
                o.w[u] = load_codes(w, at, kend);
#pragma unroll
                for (int c = 0; c < NC; c++) o.x[c][u] = load_codes(x[c], at, kend);
            }
        }
    };
    i32x4 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) acc[c] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const Batch &o) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 2 * U; u++)
#pragma unroll
            for (int c = 0; c < NC; c++)
                acc[c] = mfma16<DT>(__builtin_bit_cast(s16x8, o.w[u]), __builtin_bit_cast(s16x8, o.x[c][u]), acc[c]);
    };
    const int batches = (slice + 128 * U - 1) / (128 * U);
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
        const int n = o % NB, r = o / NB % RP, c = o / (NB * RP), at = r0 + c * RP + r;
        if (at >= t.r1 || n0 + n >= g.N) continue;
        const int row = row_of(g.c, at);
        if (row < 0) continue;
        int s = 0;
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
            for (int v = 0; v < 4; v++) s += red[v][c][p * NB + n][p * NB + r];
        const float v[1] = {(float)s * row_scale(g, at) * g.b_scale[t.e * g.b_scale_stride + n0 + n]};
        store_row<DT - kI8>(const_cast<void *>(g.c.p), (int64_t)row * g.c.ld + n0 + n, g.c_f32, v);
    }
}

// The expert of the call's row r, the last whose rows do not begin behind it: one
// after another, or, where r is the wave's and all its lanes are there, by all of
// them at once (a search's loads wait for each other).
BM_DEV int expert_of(const GemmArgs &g, int r) {
    int e = 0;
    for (int hi = g.E; hi - e > 1;) {
        const int mid = (e + hi) / 2;
        if (group_start(g, mid) <= r) e = mid;
        else hi = mid;
    }
    return e;
}
BM_DEV int wave_expert(const GemmArgs &g, int r) {
    int n = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        const int e = e0 + lane_id();
        n += __popcll(__ballot(e < g.E && group_start(g, e) <= r));
    }
    return n - 1;
}

// The parts' int32 sums (exact), scaled as in i8_epilogue.  NS parts' loads are
// issued together.
template <int DT, int NS>
__global__ void __launch_bounds__(256)
k_i8_join(GemmArgs g, const float *part, int cshift) {
    const int per = 256 >> cshift, n = ((blockIdx.x << cshift) + (threadIdx.x & ((1 << cshift) - 1))) * 8;
    const int left = min(g.N - n, 8);
    const int begin = group_start(g, 0), end = group_start(g, g.E);
    const int64_t step = (int64_t)g.R * g.N;
    for (int r = begin + blockIdx.y * per + (threadIdx.x >> cshift); r < end; r += gridDim.y * per) {
        // (before a lane leaves: all of the wave's count)
        const int e = g.E == 1 ? 0 : cshift >= 6 ? wave_expert(g, r) : expert_of(g, r);
        const int row = row_of(g.c, r);
        if (row < 0 || left <= 0) continue;
        int sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int s0 = 0; s0 < g.splits; s0 += NS) {              // (splits is a multiple of NS)
            float o[NS][8];
#pragma unroll
            for (int s = 0; s < NS; s++) load8<DT - kI8>(part, (s0 + s) * step + (int64_t)r * g.N + n, left, true, o[s]);
#pragma unroll
            for (int s = 0; s < NS; s++)
#pragma unroll
                for (int j = 0; j < 8; j++) sum[j] += __float_as_int(o[s][j]);
        }
        const float rs = row_scale(g, r);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] = (float)sum[j] * rs * g.b_scale[e * g.b_scale_stride + n + min(j, left - 1)];
        store8<DT - kI8>(const_cast<void *>(g.c.p), (int64_t)row * g.c.ld + n, left, g.c_f32, v);
    }
}

}  // namespace bm
