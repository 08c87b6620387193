// Host-side interface of the rows in 8 bits and of the products over them: the
// arguments that the C ABI's checks (rows8.cpp) hand to the launchers.
#pragma once

#include "experts_check.h"

namespace bm_host {

constexpr int kMaxK8 = (1 << 17) - 1;       // 2^14 K stays inside int32, whatever the codes

inline int row_blocks(int cols, int block) { return block ? (cols + block - 1) / block : 1; }

// a matrix of rows in 8 bits, for R rows of the call
inline int check_rows8(const bitmoe_rows8 *m, int R, int cols, bool maps) {
    if (!m) return BITMOE_EINVAL;
    const bitmoe_rows &q = m->q;
    if (q.dtype != BITMOE_I8 || q.rows < 0 || q.cols != cols || q.ld < q.cols || m->reserved != 0) return BITMOE_EINVAL;
    if (m->block != 0 && m->block != 32 && m->block != 64 && m->block != 128) return BITMOE_EINVAL;
    if (m->ld_scale < row_blocks(cols, m->block)) return BITMOE_EINVAL;
    if (q.map ? (!maps || q.div < 1 || !aligned(q.map, 4)) : q.rows < R) return BITMOE_EINVAL;
    if (R > 0 && (q.rows > 0 || !q.map) && (!q.data || !m->scale || !aligned(m->scale, 4))) return BITMOE_EINVAL;
    return BITMOE_OK;
}

int launch_quantize_rows(const bitmoe_rows &x, const bitmoe_rows8 &q, hipStream_t s);
int launch_dequantize_rows(const bitmoe_rows8 &q, const bitmoe_rows &y, hipStream_t s);
int launch_swiglu_rows8(const bitmoe_rows &gate, const bitmoe_rows &up, const bitmoe_rows8 &q, hipStream_t s);
int launch_swiglu_checkpoint(const bitmoe_rows &gate, const bitmoe_rows &up, const bitmoe_rows &h,
                             const bitmoe_rows8 &gate8, const bitmoe_rows8 &up8, hipStream_t s);
int launch_swiglu_checkpoint_backward(const bitmoe_rows &dh, const bitmoe_rows8 &gate8, const bitmoe_rows8 &up8,
                                      const bitmoe_rows &dgate, const bitmoe_rows &dup, const bitmoe_rows *h,
                                      hipStream_t s);

// y = W x in 8 bits: kForward with a and b codes, in elements (bytes) of which
// the strides and K are counted too, and their scales.  out: the outputs' type.
// The kernels are the 16-bit products': two codes lie where an element lies there.
GemmPlan i8_plan(const GemmArgs &g, bool whole);
bool i8_whole(const GemmArgs &g);            // every row begins on 16 bytes and has whole 16-byte pieces
size_t i8_ws_bytes(int E, int R, int N, int K);
// Operands laid on 16 bytes in the workspace: rows of `ld` codes (zeros behind K),
// the call's rows of x at `x` with their scales at `scale`, the experts' at `w`.
struct I8Pack {
    int64_t ld;
    size_t x, scale, w, bytes;
};
I8Pack i8_pack(int E, int R, int N, int K);
int launch_gemm_i8(int out, const GemmArgs &g, void *ws, hipStream_t s);

}  // namespace bm_host
