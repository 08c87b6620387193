// Host-side interface of the norms around a block: the arguments that the C
// ABI's checks (norm.cpp) hand to the launchers in norm_bf16.hip and norm_f16.hip.
#pragma once

#include "experts_check.h"

namespace bm_host {

constexpr int kMaxNormCols = 16384;         // a workgroup's registers hold a row
constexpr float kMinEps = 1e-30f;           // squares that vanish beside it may do so

// a matrix's first element, elements between its rows (0: one row for all) and type
struct NormMat {
    void *p;
    int64_t ld;
    bool f32;
};

struct NormArgs {
    NormMat o, gate, res, s, n;             // p NULL: not there
    const void *wa, *wb;                    // [H] or NULL
    float scale, eps;
    int32_t T, H;
};
int launch_block_norm(const NormArgs &a, int dtype, hipStream_t st);

struct NormBackArgs {
    NormMat dn, ds, s, o, gate;
    NormMat d_o, dres, dgate;               // dgate: for a gate of T rows
    const void *wa, *wb;
    float scale, eps;
    int32_t T, H;
    void *dwa, *dwb, *dg;                   // sums over tokens [H], of dw_dtype; dg: for a gate of one row, of dg_dtype
    int32_t dw_dtype, dg_dtype;
    float *partial;                         // [slices][2][H]
};
int launch_block_norm_backward(const NormBackArgs &a, int dtype, hipStream_t st);
int launch_block_norm_f16(const NormArgs &a, hipStream_t st);
int launch_block_norm_backward_f16(const NormBackArgs &a, hipStream_t st);

// The backward pass's launch: pieces of 8 columns a thread, threads of a row, rows
// of a workgroup, and workgroups, each of which leaves a slice of partial sums.  8
// columns a thread up to 2048, 16 above, in workgroups of 4 waves, or as many as a row
// needs; so many of them as run at a time (3, 2, 1 on a compute unit, by most instances'
// registers).  With a float32 stream and a gate by token 2 run where the rule takes 3:
// 16384 x 2048 183 us in its 768 slices, 149 in 512, 3001 x 2047 76 and 61; the others 92 and
// 89 (gate by channel), 119 and 110 (by token), 3001 x 2047 38 and 40, 50 and 55 (the rule
// does not know the instance).  us, 8 and 16 columns a thread: 16384 x 512 51.3 and 53.5, x 2048 96.7 and
// 101.2, x 4096 177 (a workgroup of 512 threads a compute unit) and 174 (two of 256),
// 8192 x 7168 183 (14 waves of few registers, which spill) and 169.  Above 8192 columns the
// registers spill (2048 x 16384 560 to 810).
struct NormShape {
    int pieces, nt, groups, slices;
};
inline NormShape norm_shape(int T, int H) {
    NormShape b{H <= 2048 ? 1 : 2, 0, 1, 0};
    b.nt = (H + b.pieces * 512 - 1) / (b.pieces * 512) * 64;
    b.groups = b.nt <= 128 ? 256 / b.nt : 1;
    const int most = H <= 2048 ? 768 : H <= 4096 ? 512 : 256, need = (T + b.groups - 1) / b.groups;
    b.slices = need < most ? need : most;
    return b;
}

}  // namespace bm_host
