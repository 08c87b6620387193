// Host-side interface of the norms around a block: the arguments that the C
// ABI's checks (norm.cpp) hand to the launchers in norm_kernels.hip.
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
int norm_slices(int T, int H);
int launch_block_norm_backward(const NormBackArgs &a, int dtype, hipStream_t st);

}  // namespace bm_host
