// Host-side interface of the 16-bit expert layer: the arguments that the C
// ABI's checks (experts.cpp) hand to the launchers in experts_*.hip.
#pragma once

#include "host.h"

namespace bm_host {

// Rows of a matrix.  Row r of the call is matrix row r, or map[r] / div;
// a row outside [0, rows) reads as zeros and is not written.
struct GemmRows {
    const void *p;
    const int32_t *map;
    int64_t ld;
    int32_t rows;
    uint32_t mul, shift;       // x / div = (x * mul >> 32) >> shift; mul 0: div 1
    bool span32;               // the rows a tile may read together (all, by a map; else 256) span less than 4 GiB
};

// rows of a stride of ld 16-bit elements span less than 4 GiB
inline bool span32(int rows, int64_t ld) { return ld < ((int64_t)1 << 31) && rows * ld < ((int64_t)1 << 31); }

// C[m][n] = sum_k A[m][k] B[n][k] over the groups of rows that `offsets`
// marks, in three layouts.
enum GemmLayout {
    kForward = 0,       // A = x rows (K columns),  B = W_e[n][k]:       C rows = y rows
    kGradRows = 1,      // A = dy rows (contracted), B = W_e[k][n]:      C rows = dx rows
    kGradWeights = 2,   // A = dy rows, B = x rows, contracted over the group's rows: C = dW_e[m][n]
};
struct GemmArgs {
    GemmRows a, b;             // kForward, kGradRows: b is the weights, without a map
    int64_t b_stride;          // elements between experts
    GemmRows c;                // (p is written)
    int64_t c_stride;          // kGradWeights: elements between experts
    const int32_t *offsets;    // device [E+1]; NULL: one group of R rows
    int32_t E, R;
    int32_t M, N, K;           // M: kGradWeights only (elsewhere the group's rows);
                               // K: not kGradWeights (there the group's rows)
    bool c_f32;
    bool accumulate;          // kGradWeights: add to what is there
    // epilogue: C = act(sum + bias) + res, the value before act kept in pre
    int32_t act;
    const void *bias, *res;
    void *pre;
    int64_t ld_res, ld_pre;
    bool res_f32;              // (bias and pre are of the operands' type)
    // a split contraction: `splits` parts of kper (kGradWeights: of the group's
    // rows in equal whole stages), each to its own C, c_split elements further
    int32_t splits, kper;
    int64_t c_split;
    // kGradWeights with maps: the rows they give, or -1, of each of the call's
    const int32_t *arows, *brows;
    // A (not kForward, no map) as two 16-bit parts of a half of each value
    // (split16): the second's elements `a_low` further than the first's; 0: one
    int64_t a_low;
    // products in 8 bits (launch_gemm_i8): a and b are codes; the sum is taken
    // times a_scale[matrix row * a_ld_scale] and b_scale[e * b_scale_stride + n], or,
    // with raw, left as the int32 it is (a part of a split contraction)
    const float *a_scale, *b_scale;
    int64_t a_ld_scale, b_scale_stride;
    bool raw;
};

// How a product runs: which kernel, its tiles, into how many parts the
// contraction is split.  A rule on the sizes the host knows.
enum GemmKind { kAny, kTile256, kTile128x256, kTile128, kTile64x128, kFew };
struct GemmPlan {
    int kind;
    int mt, nt;         // row tiles (of all groups, at most; kGradWeights: of an expert), column tiles
    int splits, kper;
    int64_t grid;       // workgroups that would take one tile each
    int parts, chunks;  // kFew: its P and NC
    size_t ws;          // bytes: the parts' float32, then (kGradWeights) the rows of both maps
    bool pack;          // 8 bits: the operands' rows are laid on 16 bytes first (behind the parts in ws)
};
// every row begins on a 16-byte address and has whole 8-element pieces
bool gemm_whole(int layout, const GemmArgs &g);
GemmPlan gemm_plan(int layout, const GemmArgs &g, bool whole);
// the row and column tiles and the grid of tiles of bm x bn (p->splits parts)
void plan_tiles(int layout, const GemmArgs &g, int bm, int bn, GemmPlan *p);
// workspace of a product of these sizes, whatever its addresses
size_t gemm_ws_bytes(int layout, const GemmArgs &g);
int launch_gemm(int layout, int dtype, const GemmArgs &g, void *ws, hipStream_t s);
int launch_experts_fwd(int dtype, const GemmArgs &g, const GemmPlan &p, hipStream_t s);
int launch_experts_dx(int dtype, const GemmArgs &g, const GemmPlan &p, hipStream_t s);
int launch_experts_dw(int dtype, const GemmArgs &g, const GemmPlan &p, hipStream_t s);

// dz = dy act'(pre) (dz may be NULL) and, with db, its column sums by slices
// of rows (partial [slices][N]); low: dz in two parts, the second's that many
// elements further (0: rounded to one)
struct ActBackward {
    const void *dy, *pre;
    void *dz;
    int64_t ld_dy, ld_pre, ld_dz, low;
    int32_t T, N, act;
    void *db;
    int32_t db_dtype;
    float *partial;
};
int act_backward_slices(int T, int N);
int launch_act_backward(const ActBackward &p, int dtype, hipStream_t s);

// rows of c that the call's rows of no group go to: 0
int launch_clear_ungrouped(const int32_t *offsets, int E, int R, const GemmRows &c, int cols, bool f32, hipStream_t s);
int launch_swiglu(const bitmoe_rows &gate, const bitmoe_rows &up, const bitmoe_rows &h, int dtype, hipStream_t s);
int launch_swiglu_backward(const bitmoe_rows &dh, const bitmoe_rows &gate, const bitmoe_rows &up,
                           const bitmoe_rows &dgate, const bitmoe_rows &dup, int dtype, hipStream_t s);
int launch_combine(const bitmoe_rows &o, const float *w, int T, int k, const bitmoe_rows *residual,
                   const bitmoe_rows &y, hipStream_t s);
int launch_combine_backward(const bitmoe_rows &dy, const bitmoe_rows *o, const float *w, int T, int k,
                            const bitmoe_rows *d_o, float *dw, int dtype, hipStream_t s);

}  // namespace bm_host
