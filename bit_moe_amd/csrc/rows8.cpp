// C ABI of the rows in 8 bits: host-side validation, as in experts.cpp (every
// check runs before the first launch).
#include "rows8.h"

namespace {

using namespace bm_host;

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

// gate and up of one 16-bit type
int check_gates(const bitmoe_rows *gate, const bitmoe_rows *up) {
    if (!gate) return BITMOE_EINVAL;
    const int rc = check_sizes(1, gate->rows, gate->cols, 1);
    if (rc) return rc;
    if (!is16(gate->dtype) || check_rows(gate, gate->rows, gate->cols, false)) return BITMOE_EINVAL;
    if (check_rows(up, gate->rows, gate->cols, false) || up->dtype != gate->dtype) return BITMOE_EINVAL;
    return BITMOE_OK;
}

}  // namespace

extern "C" {

int moe_quantize_rows(const bitmoe_rows *x, const bitmoe_rows8 *q, void *stream) {
    if (!x) return BITMOE_EINVAL;
    int rc = check_sizes(1, x->rows, x->cols, 1);
    if (rc || (rc = check_rows(x, x->rows, x->cols, false)) || (rc = check_rows8(q, x->rows, x->cols, false))) return rc;
    if (x->rows == 0) return BITMOE_OK;
    return launch_quantize_rows(*x, *q, as_stream(stream));
}

int moe_dequantize_rows(const bitmoe_rows8 *q, const bitmoe_rows *y, void *stream) {
    if (!q) return BITMOE_EINVAL;
    int rc = check_sizes(1, q->q.rows, q->q.cols, 1);
    if (rc || (rc = check_rows8(q, q->q.rows, q->q.cols, false)) || (rc = check_rows(y, q->q.rows, q->q.cols, false)))
        return rc;
    if (q->q.rows == 0) return BITMOE_OK;
    return launch_dequantize_rows(*q, *y, as_stream(stream));
}

int moe_swiglu_rows8(const bitmoe_rows *gate, const bitmoe_rows *up, const bitmoe_rows8 *q, void *stream) {
    int rc = check_gates(gate, up);
    if (rc || (rc = check_rows8(q, gate->rows, gate->cols, false))) return rc;
    if (gate->rows == 0) return BITMOE_OK;
    return launch_swiglu_rows8(*gate, *up, *q, as_stream(stream));
}

int moe_swiglu_checkpoint(const bitmoe_rows *gate, const bitmoe_rows *up, const bitmoe_rows *h,
                          const bitmoe_rows8 *gate8, const bitmoe_rows8 *up8, void *stream) {
    int rc = check_gates(gate, up);
    if (rc) return rc;
    const int R = gate->rows, I = gate->cols;
    if (check_rows(h, R, I, false) || h->dtype != gate->dtype) return BITMOE_EINVAL;
    if (check_rows8(gate8, R, I, false) || check_rows8(up8, R, I, false)) return BITMOE_EINVAL;
    if (gate8->block == 0 || up8->block != gate8->block) return BITMOE_EINVAL;
    if (R == 0) return BITMOE_OK;
    return launch_swiglu_checkpoint(*gate, *up, *h, *gate8, *up8, as_stream(stream));
}

int moe_swiglu_checkpoint_backward(const bitmoe_rows *dh, const bitmoe_rows8 *gate8, const bitmoe_rows8 *up8,
                                   const bitmoe_rows *dgate, const bitmoe_rows *dup, const bitmoe_rows *h,
                                   void *stream) {
    if (!dh) return BITMOE_EINVAL;
    const int R = dh->rows, I = dh->cols, dt = dh->dtype;
    const int rc = check_sizes(1, R, I, 1);
    if (rc) return rc;
    if (!is16(dt) || check_rows(dh, R, I, false)) return BITMOE_EINVAL;
    if (check_rows8(gate8, R, I, false) || check_rows8(up8, R, I, false)) return BITMOE_EINVAL;
    if (gate8->block == 0 || up8->block != gate8->block) return BITMOE_EINVAL;
    for (const bitmoe_rows *m : {dgate, dup})
        if (check_rows(m, R, I, false) || m->dtype != dt) return BITMOE_EINVAL;
    if (h && (check_rows(h, R, I, false) || h->dtype != dt)) return BITMOE_EINVAL;
    if (R == 0) return BITMOE_OK;
    return launch_swiglu_checkpoint_backward(*dh, *gate8, *up8, *dgate, *dup, h, as_stream(stream));
}

size_t moe_expert_matmul_i8_workspace_bytes(int E, int R, int N, int K) {
    if (check_sizes(E, R, N, K) || K > kMaxK8) return 0;
    return i8_ws_bytes(E, R, N, K);
}

int moe_expert_matmul_i8(const bitmoe_rows8 *x, const bitmoe_experts8 *w, const int32_t *offsets, int R,
                         const bitmoe_rows *y, void *ws, size_t ws_bytes, void *stream) {
    if (!x || !w) return BITMOE_EINVAL;
    const bitmoe_experts &q = w->q;
    int rc = check_sizes(q.E, R, q.N, q.K);
    if (rc) return rc;
    if (q.K > kMaxK8) return BITMOE_EUNSUPPORTED;
    if (q.dtype != BITMOE_I8 || q.ld < q.K || (q.E > 1 && q.stride < (int64_t)(q.N - 1) * q.ld + q.K)) return BITMOE_EINVAL;
    if (!q.data || !w->scale || !aligned(w->scale, 4) || (q.E > 1 && w->scale_stride < q.N)) return BITMOE_EINVAL;
    if ((rc = check_rows8(x, R, q.K, true)) || (rc = check_rows(y, R, q.N, true))) return rc;
    if (x->block != 0) return BITMOE_EINVAL;
    if (offsets ? !aligned(offsets, 4) : q.E != 1) return BITMOE_EINVAL;
    if (R == 0) return BITMOE_OK;
    const size_t need = i8_ws_bytes(q.E, R, q.N, q.K);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return BITMOE_EWORKSPACE;
    GemmArgs g{};
    g.a = rows_arg(&x->q);
    g.b = GemmRows{q.data, nullptr, q.ld, q.N, 0, 0, false};
    g.c = rows_arg(y);
    g.b_stride = q.stride;
    g.offsets = offsets;
    g.E = q.E;
    g.R = R;
    g.N = q.N;
    g.K = q.K;
    g.c_f32 = y->dtype == BITMOE_F32;
    g.a_scale = x->scale;
    g.a_ld_scale = x->ld_scale;
    g.b_scale = w->scale;
    g.b_scale_stride = w->scale_stride;
    return launch_gemm_i8(y->dtype, g, ws, as_stream(stream));
}

}  // extern "C"
