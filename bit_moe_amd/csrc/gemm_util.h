// Device helpers of the 16-bit matrix products: element types, tiles in LDS,
// matrix-core operands, the search for a workgroup's tile, the epilogue.
#pragma once

#include "common.h"
#include "experts.h"

namespace bm {

using bm_host::GemmArgs;
using bm_host::GemmRows;
using bm_host::kForward;
using bm_host::kGradRows;
using bm_host::kGradWeights;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr int kBK = 64;             // contraction per stage

// ---- elements -------------------------------------------------------------
// DT: BITMOE_BF16 or BITMOE_F16
template <int DT>
BM_DEV f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c) {
    if constexpr (DT == BITMOE_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                      0, 0, 0);
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
template <int DT>
BM_DEV float elem_f32(uint32_t bits) { return DT == BITMOE_BF16 ? bf16_to_f32(bits) : fp16_to_f32(bits); }
// two values rounded to nearest, the first in the low half
template <int DT>
BM_DEV uint32_t elem_pair(float a, float b) {
    if constexpr (DT == BITMOE_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2_t));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2_t));
}

// A value in fp32 as two 16-bit ones for the matrix cores, which take no more:
// a half of it rounded, and what that leaves, 2^8 (bfloat16) or 2^11 (float16)
// times, so that v = 2 (high + low / low_scale).  What both leave is at most
// 2^-16 (2^-22) of v or, in float16, 2^-35; the half keeps float16's largest
// values from its infinity, and the low part's scale its smallest from zero.
template <int DT>
constexpr float low_scale() { return DT == BITMOE_BF16 ? 256.f : 2048.f; }
template <int DT>
BM_DEV void split16(const float (&v)[8], float (&high)[8], float (&low)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const uint32_t h = elem_pair<DT>(0.5f * v[j], 0.5f * v[j + 1]);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            high[j + i] = elem_f32<DT>(h >> (16 * i) & 0xFFFFu);
            const float left = 0.5f * v[j + i] - high[j + i];
            low[j + i] = fabsf(high[j + i]) < INFINITY ? left * low_scale<DT>() : 0.f;
        }
    }
}

// 16 bytes at any element's address: gfx950 reads and writes global
// memory at any alignment, so rows need not be aligned to a vector
struct __attribute__((packed, aligned(2))) U128 { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) F128 { float w[4]; };

BM_DEV uint4 load16(const uint16_t *p) {
    const U128 u = *reinterpret_cast<const U128 *>(p);
    return make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
}
// elements [0, n) of 8, the rest zero
BM_DEV uint4 load16_part(const uint16_t *p, int n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < n) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// eight consecutive values of a row of DT or fp32, the first n of them (n >= 1;
// the rest 0)
BM_DEV void load4_f32(const float *q, int n, float *v) {
    if (n >= 4) {
        const F128 u = *reinterpret_cast<const F128 *>(q);
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = u.w[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = j < n ? q[j] : 0.f;
    }
}
template <int DT>
BM_DEV void load8(const void *p, int64_t i, int n, bool f32, float *v) {
    if (f32) {
        const float *q = static_cast<const float *>(p) + i;
        load4_f32(q, n, v);
        load4_f32(q + 4, n - 4, v + 4);
        return;
    }
    const uint16_t *q = static_cast<const uint16_t *>(p) + i;
    const uint4 u = n >= 8 ? load16(q) : load16_part(q, n);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = elem_f32<DT>(w[j >> 1] >> (16 * (j & 1)) & 0xFFFFu);
}
template <int DT>
BM_DEV void store8(void *p, int64_t i, int n, bool f32, const float *v) {
    if (f32) {
        float *q = static_cast<float *>(p) + i;
        if (n >= 8) {
            *reinterpret_cast<F128 *>(q) = F128{{v[0], v[1], v[2], v[3]}};
            *reinterpret_cast<F128 *>(q + 4) = F128{{v[4], v[5], v[6], v[7]}};
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j < n) q[j] = v[j];
        }
        return;
    }
    uint16_t *q = static_cast<uint16_t *>(p) + i;
    U128 u;
#pragma unroll
    for (int j = 0; j < 4; j++) u.w[j] = elem_pair<DT>(v[2 * j], v[2 * j + 1]);
    if (n >= 8) {
        *reinterpret_cast<U128 *>(q) = u;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) q[j] = (uint16_t)(u.w[j >> 1] >> (16 * (j & 1)));
    }
}

// eight values, or one
template <int DT>
BM_DEV void load_row(const void *p, int64_t i, bool f32, float (&v)[8]) { load8<DT>(p, i, 8, f32, v); }
template <int DT>
BM_DEV void store_row(void *p, int64_t i, bool f32, const float (&v)[8]) { store8<DT>(p, i, 8, f32, v); }
template <int DT>
BM_DEV void load_row(const void *p, int64_t i, bool f32, float (&v)[1]) {
    v[0] = f32 ? static_cast<const float *>(p)[i] : elem_f32<DT>(static_cast<const uint16_t *>(p)[i]);
}
template <int DT>
BM_DEV void store_row(void *p, int64_t i, bool f32, const float (&v)[1]) {
    if (f32) static_cast<float *>(p)[i] = v[0];
    else static_cast<uint16_t *>(p)[i] = (uint16_t)elem_pair<DT>(v[0], 0.f);
}

// ---- rows and groups ------------------------------------------------------
// m / div for 0 <= m < 2^31 (the multiplier and shift of rows_arg)
BM_DEV int divided(const GemmRows &q, int m) { return q.mul ? (int)(__umulhi((uint32_t)m, q.mul) >> q.shift) : m; }
// matrix row of the call's row r, or -1
BM_DEV int row_of(const GemmRows &q, int r) {
    int m = r;
    if (q.map) {
        m = q.map[r];
        if (m < 0) return -1;
        m = divided(q, m);
    }
    return m < q.rows ? m : -1;
}
// first row of group e (and of e + 1: its end), kept inside the call's rows
BM_DEV int group_start(const GemmArgs &g, int e) {
    if (!g.offsets) return e ? g.R : 0;
    return min(max(g.offsets[e], 0), g.R);
}

struct Tile {
    int e, r0, r1;      // expert, its rows
    int m, n;           // tile indexes
};

// The tiles of a workgroup.  Workgroups go round the 8 XCDs in turn; each XCD
// has its own list of tiles, whose neighbours share operands through its L2,
// and its workgroups take them in order.
//  Rows (forward, rows' gradient): the (expert, row tile, column tile) of all
//   groups, one after another, 8 row tiles by all column tiles at a time, are
//   cut into 8 runs.  Every wave counts the groups' row tiles by itself: each
//   lane those of a run of experts, and a scan over the lanes places them.
//  Weights' gradient: the tiles are fixed, their work (a group's rows) is not:
//   each XCD takes an eighth of every expert's tiles.
__host__ __device__ inline int dw_eighth(int mt, int nt) { return (mt * nt + 7) / 8; }

template <int LAY, int BM>
struct Tiles {
    int xcd, slot, step;       // the next tile's place in the XCD's list
    int per, mine, incl;       // rows: experts a lane counts, their row tiles, with all lanes' before
    int mt, nt;                // dw: row tiles; column tiles
    int64_t items, per_xcd;

    BM_DEV void init(const GemmArgs &g, int mtiles, int ntiles, int bid, int grid) {
        xcd = bid & 7;
        slot = bid >> 3;
        step = grid >> 3;
        mt = mtiles;
        nt = ntiles;
        if (LAY == kGradWeights) return;
        const int lane = lane_id();
        per = (g.E + 63) / 64;
        mine = 0;
        for (int i = 0; i < per; i++) {
            const int e = lane * per + i;
            if (e < g.E) mine += (max(group_start(g, e + 1) - group_start(g, e), 0) + BM - 1) / BM;
        }
        incl = mine;
        if (g.E == 1) incl = __builtin_amdgcn_readfirstlane(mine);
        else
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(incl, o, kWave);
                if (lane >= o) incl += v;
            }
        items = (int64_t)__builtin_amdgcn_readlane(incl, 63) * nt;
        per_xcd = (items + 7) / 8;
    }
    BM_DEV bool next(const GemmArgs &g, Tile *t) {
        const int at = slot;
        slot += step;
        int idx, cnt;
        if (LAY == kGradWeights) {
            const int n8 = dw_eighth(mt, nt);
            t->e = at / n8;
            idx = xcd * n8 + at - t->e * n8;
            cnt = mt;
            if (t->e >= g.E) return false;
            if (idx >= mt * nt) {                  // the eighths are not whole: none here
                t->m = -1;
                return true;
            }
            t->r0 = __builtin_amdgcn_readfirstlane(group_start(g, t->e));
            t->r1 = max(__builtin_amdgcn_readfirstlane(group_start(g, t->e + 1)), t->r0);
        } else {
            const int64_t item = xcd * per_xcd + at;
            if (at >= per_xcd || item >= items) return false;
            const int place = (int)(item / nt);                          // among the row tiles
            const int src = __builtin_ctzll(__ballot(place < incl));     // the lane whose run holds it
            int base = __builtin_amdgcn_readlane(incl - mine, src), e = src * per, r0, r1;
            for (;; e++) {
                r0 = group_start(g, e);
                r1 = group_start(g, e + 1);
                cnt = (max(r1 - r0, 0) + BM - 1) / BM;
                if (place < base + cnt || e >= g.E - 1) break;
                base += cnt;
            }
            idx = (int)(item - (int64_t)base * nt);
            t->e = __builtin_amdgcn_readfirstlane(e);
            t->r0 = __builtin_amdgcn_readfirstlane(r0);
            t->r1 = __builtin_amdgcn_readfirstlane(r1);
        }
        const int blk = idx / (8 * nt), mb = min(8, cnt - 8 * blk), rem = idx - blk * 8 * nt;
        t->m = __builtin_amdgcn_readfirstlane(8 * blk + rem % mb);
        t->n = __builtin_amdgcn_readfirstlane(rem / mb);
        return true;
    }
};

// The part of the contraction that a tile takes: [beg, end) of it, and which
// part it is (the column tiles of the list are those of the parts, one part
// after another).  Weights' gradient: the group's rows become the part's.
struct Span {
    int beg, end, split;
};
template <int LAY>
BM_DEV Span span_of(const GemmArgs &g, Tile *t, int nt) {
    Span k{0, LAY == kGradWeights ? t->r1 - t->r0 : g.K, 0};
    if (g.splits > 1) {
        k.split = t->n / nt;
        t->n -= k.split * nt;
        if (LAY == kGradWeights) {
            const int per = ((k.end + kBK - 1) / kBK + g.splits - 1) / g.splits * kBK;
            const int r0 = min(t->r0 + k.split * per, t->r1);
            t->r1 = min(r0 + per, t->r1);
            t->r0 = r0;
            k.end = t->r1 - r0;
        } else {
            k.beg = min(k.split * g.kper, g.K);
            k.end = min(k.beg + g.kper, g.K);
        }
    }
    return k;
}

// ---- tiles in LDS ---------------------------------------------------------
// An operand's stage is X rows of kBK elements (contiguous along the
// contraction: KC) or kBK rows of X elements (KS), in 16-byte pieces.
//  KC: piece c of row r at slot c ^ swz(r) of the row's pieces, so that the
//      16-byte reads of consecutive rows, one piece each, run without bank
//      conflicts (measured: 4.4 cycles for a wave's 1 KiB; rows padded by 16
//      bytes take 8.2, rows neither padded nor swizzled 16.2).
//  KS: pieces move in pairs of 32 bytes, pair c of row k at c ^ swz(k): a
//      transposed read takes 32 bytes of each of 4 consecutive rows (8, 16, 24
//      rows further for the wave's other lanes), and these fall on different
//      banks too.
BM_DEV int kc_swz(int r) { return r & 7; }
template <int X>
BM_DEV int ks_swz(int k) {
    return X >= 128 ? (k & 3) | ((k >> 1) & 4) : (k & 3);
}
// piece p of the stage (in LDS order): its row and its piece in the row
template <bool KC, int X>
BM_DEV void piece_at(int p, int *row, int *col) {
    if (KC) {
        *row = p / (kBK / 8);
        *col = p % (kBK / 8) ^ kc_swz(*row);
    } else {
        *row = p / (X / 8);
        const int s = p % (X / 8);
        *col = ((s >> 1) ^ ks_swz<X>(*row)) << 1 | (s & 1);
    }
}
// the wave's matrix-core operand: 16 rows (KC) or columns (KS) from x0, 32 of
// the contraction from kk; lane l holds row l % 16, contraction 8 (l / 16) + j
template <bool KC, int X>
BM_DEV s16x8 frag(const uint16_t *tile, int x0, int kk, int lane) {
    const int i = lane & 15, q = lane >> 4;
    if (KC) {
        const int row = x0 + i;
        return *reinterpret_cast<const s16x8 *>(tile + row * kBK + ((((kk >> 3) + q) ^ kc_swz(row)) << 3));
    } else {
        // a transposing read: 16 lanes give 4 rows of 16 elements, four lanes
        // a row, and receive the 16 columns, 4 elements each
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int k = kk + 8 * q + (i >> 2);
        const uint16_t *p = tile + k * X + (((x0 >> 4) ^ ks_swz<X>(k)) << 4) + ((i & 3) << 2);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * X));
        return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
}

// ---- epilogue -------------------------------------------------------------
BM_DEV float act_fwd(float z, int act) {
    switch (act) {
        case BITMOE_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
        // (1 + erf of a negative number is erfc of the positive one, which keeps the
        // digits that the sum cancels: all of them below z = -5.5)
        case BITMOE_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);
        case BITMOE_ACT_GELU_TANH: {
            // 0.5 (1 + tanh u) = 1 / (1 + e^-2u)
            const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
            return z / (1.f + __expf(-2.f * u));
        }
        case BITMOE_ACT_SILU: return z / (1.f + __expf(-z));
        default: return z;
    }
}

template <int W>
BM_DEV void act_row(float (&v)[W], int act) {
#define BM_ACT(A)                                                   \
    case A:                                                         \
        _Pragma("unroll") for (int j = 0; j < W; j++) v[j] = act_fwd(v[j], A); \
        break;
    switch (act) {
        BM_ACT(BITMOE_ACT_RELU)
        BM_ACT(BITMOE_ACT_GELU)
        BM_ACT(BITMOE_ACT_GELU_TANH)
        BM_ACT(BITMOE_ACT_SILU)
    }
#undef BM_ACT
}
// d act / dz
BM_DEV float act_slope(float z, int act) {
    switch (act) {
        case BITMOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case BITMOE_ACT_GELU:
            return 0.5f * erfcf(z * -0.70710678118654752f) + z * 0.39894228040143268f * __expf(-0.5f * z * z);
        case BITMOE_ACT_GELU_TANH: {
            // with p = 1 / (1 + e^-2u): p + 2 z p (1 - p) du/dz; p is 0 or 1 long
            // before |z| = 16, and z^2 may not be infinite beside it
            z = z > 16.f ? 16.f : z < -16.f ? -16.f : z;
            const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z), p = 1.f / (1.f + __expf(-2.f * u));
            return p + 2.f * z * p * (1.f - p) * 0.79788456080286536f * (1.f + 0.134145f * z * z);
        }
        case BITMOE_ACT_SILU: {
            const float p = 1.f / (1.f + __expf(-z));
            return p + z * p * (1.f - p);
        }
        default: return 1.f;
    }
}

BM_DEV void slope_row(float (&d)[8], const float (&z)[8], int act) {
#define BM_SLOPE(A)                                                                     \
    case A:                                                                             \
        _Pragma("unroll") for (int j = 0; j < 8; j++) d[j] *= act_slope(z[j], A);       \
        break;
    switch (act) {
        BM_SLOPE(BITMOE_ACT_RELU)
        BM_SLOPE(BITMOE_ACT_GELU)
        BM_SLOPE(BITMOE_ACT_GELU_TANH)
        BM_SLOPE(BITMOE_ACT_SILU)
    }
#undef BM_SLOPE
}

// Eight (W = 8) outputs of a row, or the one at the edge (W = 1): n.. of row
// `row` of the output, with the bias's and the residual's values;
// part: where a part of a split begins.
template <int LAY, int DT, int W>
BM_DEV void finish(const GemmArgs &g, int e, int64_t part, int row, int n, float (&v)[W], const float (&bias)[W],
                   const float (&res)[W]) {
    int64_t at = part + (int64_t)row * g.c.ld + n;
    if constexpr (LAY == kGradWeights) {
        at += (int64_t)e * g.c_stride;
        if (g.accumulate) {
            float o[W];
            load_row<DT>(g.c.p, at, g.c_f32, o);
#pragma unroll
            for (int j = 0; j < W; j++) v[j] += o[j];
        }
    }
    if constexpr (LAY == kForward) {
        if (g.bias) {
#pragma unroll
            for (int j = 0; j < W; j++) v[j] += bias[j];
        }
        if (g.pre) store_row<DT>(g.pre, (int64_t)row * g.ld_pre + n, false, v);
        if (g.act != BITMOE_ACT_NONE) act_row(v, g.act);
        if (g.res) {
#pragma unroll
            for (int j = 0; j < W; j++) v[j] += res[j];
        }
    }
    store_row<DT>(const_cast<void *>(g.c.p), at, g.c_f32, v);
}

// the output row of each of a tile's rows, or -1
template <int LAY, int BM>
BM_DEV void set_rows(const GemmArgs &g, const Tile &t, int m0, int tid, int *srow) {
    if (tid < BM) {
        const int m = m0 + tid;
        srow[tid] = LAY == kGradWeights ? (m < g.M ? m : -1) : m < t.r1 - t.r0 ? row_of(g.c, t.r0 + m) : -1;
    }
}

// The waves' accumulators to memory.  A lane holds 4 columns of one row of
// each 16 x 16 product; through LDS (a wave's own part of `lds`) it takes 8
// columns, 16 rows by half the wave's columns at a time.
// The wave's rows and columns come in HALVES equal runs, its own part of each
// of the tile's halves of BM and BN: run h of rows at h * BM / 2 + m_at.  srow:
// the output row of each of the tile's rows, or -1.
// Where there is nothing to add and the tile ends inside the matrix, the code
// is unrolled.  Else the pass over the rows is a loop whose end moves the
// accumulators down, one copy of that much longer code and no register indexed;
// the moves alone take 4 us a tile of 256 x 256, so the short form is worth its
// code.
// Lanes hand values to each other through LDS between these points: the wave's
// LDS operations run in order, and the point keeps the compiler from letting
// some lanes run ahead (it may otherwise give lanes without a row a path of
// their own through the passes, whose writes then overtake the others' reads).
BM_DEV void wave_together() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int TN>
constexpr int epilogue_floats() { return 16 * (8 * TN + 4); }       // a wave's part

template <int LAY, int DT, int BM, int BN, int HALVES, int TM, int TN>
BM_DEV void tile_epilogue(const GemmArgs &g, f32x4 (&acc)[TM][TN], float *lds, const int *srow, int e, int split,
                          int n0, int m_at, int n_at, int wave, int lane) {
    constexpr int MR = 16 * TM / HALVES, TH = TN / 2, CW = 16 * TH;      // columns at a time
    constexpr int LDW = CW + 4, LPR = CW / 8, RPI = 64 / LPR, IT = 16 / RPI;
    static_assert(TN % 2 == 0 && (HALVES == 2 || HALVES == 1), "");
    float *sw = lds + wave * epilogue_floats<TN>();
    const int r0 = lane / LPR, c = (lane % LPR) * 8;
    const int nn[2] = {n0 + n_at + c, n0 + n_at + c + (HALVES == 2 ? BN / 2 : CW)};
    auto out_row = [&](int m) { return srow[m / MR * (BM / 2) + m_at + m % MR]; };
    const bool has_res = LAY == kForward && g.res;

    const bool plain = LAY == kForward ? !g.bias && !g.pre && !g.res && g.act == BITMOE_ACT_NONE : !g.accumulate;
    if (plain && n0 + BN <= g.N) {
        char *out = static_cast<char *>(const_cast<void *>(g.c.p));
        const int es = g.c_f32 ? 4 : 2;
        if (LAY == kGradWeights) out += (int64_t)e * g.c_stride * es;
        out += split * g.c_split * es;
#pragma unroll
        for (int q = 0; q < TM; q++) {
            int rows[IT];
#pragma unroll
            for (int it = 0; it < IT; it++) rows[it] = out_row(16 * q + it * RPI + r0);
#pragma unroll
            for (int h = 0; h < 2; h++) {
#pragma unroll
                for (int j = 0; j < TH; j++)
                    *reinterpret_cast<f32x4 *>(sw + (lane & 15) * LDW + 16 * j + 4 * (lane >> 4)) = acc[q][h * TH + j];
                wave_together();
#pragma unroll
                for (int it = 0; it < IT; it++) {
                    const int r = it * RPI + r0;
                    const f32x4 a = *reinterpret_cast<const f32x4 *>(sw + r * LDW + c);
                    const f32x4 b = *reinterpret_cast<const f32x4 *>(sw + r * LDW + c + 4);
                    if (rows[it] < 0) continue;
                    char *p = out + ((int64_t)rows[it] * g.c.ld + nn[h]) * es;
                    if (g.c_f32) {
                        reinterpret_cast<F128 *>(p)[0] = F128{{a[0], a[1], a[2], a[3]}};
                        reinterpret_cast<F128 *>(p)[1] = F128{{b[0], b[1], b[2], b[3]}};
                    } else {
                        *reinterpret_cast<U128 *>(p) = U128{{elem_pair<DT>(a[0], a[1]), elem_pair<DT>(a[2], a[3]),
                                                             elem_pair<DT>(b[0], b[1]), elem_pair<DT>(b[2], b[3])}};
                    }
                }
                wave_together();
            }
        }
        return;
    }
    auto residual = [&](int q, int h, int it, float (&r)[8]) {
        const int row = out_row(16 * q + it * RPI + r0);
        if (has_res && row >= 0 && nn[h] + 8 <= g.N)
            load_row<DT>(g.res, (int64_t)row * g.ld_res + nn[h], g.res_f32, r);
    };
    // (the residual one pass ahead of its use)
    float res[2][IT][8], ahead[2][IT][8], bias[2][8];
    if (LAY == kForward) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (g.bias && nn[h] + 8 <= g.N) load_row<DT>(g.bias, nn[h], false, bias[h]);
#pragma unroll
            for (int it = 0; it < IT; it++) residual(0, h, it, res[h][it]);
        }
    }
#pragma unroll 1
    for (int q = 0; q < TM; q++) {
        if (LAY == kForward && q + 1 < TM) {
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int it = 0; it < IT; it++) residual(q + 1, h, it, ahead[h][it]);
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int j = 0; j < TH; j++)
                *reinterpret_cast<f32x4 *>(sw + (lane & 15) * LDW + 16 * j + 4 * (lane >> 4)) = acc[0][h * TH + j];
            wave_together();
#pragma unroll
            for (int it = 0; it < IT; it++) {
                const int r = it * RPI + r0, row = out_row(16 * q + r), left = g.N - nn[h];
                if (row >= 0 && left >= 8) {
                    const f32x4 a = *reinterpret_cast<const f32x4 *>(sw + r * LDW + c);
                    const f32x4 b = *reinterpret_cast<const f32x4 *>(sw + r * LDW + c + 4);
                    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                    finish<LAY, DT>(g, e, split * g.c_split, row, nn[h], v, bias[h], res[h][it]);
                } else if (row >= 0) {
#pragma unroll 1
                    for (int j = 0; j < left; j++) {
                        float v[1] = {sw[r * LDW + c + j]}, one[1] = {0.f}, bi[1] = {0.f};
                        if (LAY == kForward && g.bias) load_row<DT>(g.bias, nn[h] + j, false, bi);
                        if (has_res) load_row<DT>(g.res, (int64_t)row * g.ld_res + nn[h] + j, g.res_f32, one);
                        finish<LAY, DT>(g, e, split * g.c_split, row, nn[h] + j, v, bi, one);
                    }
                }
            }
            wave_together();
        }
        if (LAY == kForward) {
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int it = 0; it < IT; it++)
#pragma unroll
                    for (int j = 0; j < 8; j++) res[h][it][j] = ahead[h][it][j];
        }
#pragma unroll
        for (int i = 0; i + 1 < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++) acc[i][j] = acc[i + 1][j];
    }
}

}  // namespace bm
