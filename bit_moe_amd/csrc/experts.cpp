// C ABI of the 16-bit expert layer: host-side validation and launch
// orchestration, as in api.cpp (every check runs before the first launch).
#include <algorithm>
#include <cstdint>

#include "experts_check.h"

namespace {

using namespace bm_host;

constexpr size_t kAlign = 256;

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }
inline size_t up256(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

int check_experts(const bitmoe_experts *w, int R) {
    if (!w) return BITMOE_EINVAL;
    const int rc = check_sizes(w->E, R, w->N, w->K);
    if (rc) return rc;
    if (w->ld < w->K || (w->E > 1 && w->stride < (int64_t)(w->N - 1) * w->ld + w->K)) return BITMOE_EINVAL;
    if (!is16(w->dtype) && w->dtype != BITMOE_F32) return BITMOE_EINVAL;
    if (!w->data || !aligned(w->data, esize(w->dtype))) return BITMOE_EINVAL;
    return BITMOE_OK;
}

int check_ws(void *ws, size_t have, size_t need) {
    if (need == 0) return BITMOE_OK;
    if (!ws || have < need || !aligned(ws, kAlign)) return BITMOE_EWORKSPACE;
    return BITMOE_OK;
}

GemmRows weights_arg(const bitmoe_experts *w) {
    return GemmRows{w->data, nullptr, w->ld, w->N, 0, 0, span32(256, w->ld)};
}

// y = W x or dx = W^T dy over groups
GemmArgs rows_product(const bitmoe_rows *a, const bitmoe_experts *w, const int32_t *offsets, int R,
                      const bitmoe_rows *c, bool dx) {
    GemmArgs g{};
    g.a = rows_arg(a);
    g.b = weights_arg(w);
    g.b_stride = w->stride;
    g.c = rows_arg(c);
    g.offsets = offsets;
    g.E = w->E;
    g.R = R;
    g.N = dx ? w->K : w->N;
    g.K = dx ? w->N : w->K;
    g.c_f32 = c->dtype == BITMOE_F32;
    return g;
}

GemmArgs weights_product(const bitmoe_rows *dy, const bitmoe_rows *x, const int32_t *offsets, int R,
                         const bitmoe_experts *dw, int accumulate) {
    GemmArgs g{};
    g.a = rows_arg(dy);
    g.b = rows_arg(x);
    g.c = weights_arg(dw);
    g.c_stride = dw->stride;
    g.offsets = offsets;
    g.E = dw->E;
    g.R = R;
    g.M = dw->N;
    g.N = dw->K;
    g.c_f32 = dw->dtype == BITMOE_F32;
    g.accumulate = accumulate != 0;
    return g;
}

int expert_rows_product(const bitmoe_rows *a, const bitmoe_experts *w, const int32_t *offsets, int R,
                        const bitmoe_rows *c, void *ws, size_t ws_bytes, void *stream, bool dx) {
    int rc = check_experts(w, R);
    if (rc) return rc;
    if ((rc = check_rows(a, R, dx ? w->N : w->K, true)) || (rc = check_rows(c, R, dx ? w->K : w->N, true))) return rc;
    if (!is16(w->dtype) || a->dtype != w->dtype || !out_type(c->dtype, w->dtype)) return BITMOE_EINVAL;
    if (R == 0) return BITMOE_OK;
    if (!offsets || !aligned(offsets, 4)) return BITMOE_EINVAL;
    const GemmArgs g = rows_product(a, w, offsets, R, c, dx);
    const int layout = dx ? kGradRows : kForward;
    if ((rc = check_ws(ws, ws_bytes, gemm_ws_bytes(layout, g)))) return rc;
    return launch_gemm(layout, w->dtype, g, ws, as_stream(stream));
}

// dz (two parts of whole 16-byte pieces a row), db's partial sums and the
// products' own, in moe_linear_backward's workspace, whatever the call wants
struct BackwardWs {
    size_t dz, db, gemm, bytes;
};
int64_t part_cols(int N) { return (N + 7) / 8 * 8; }
BackwardWs backward_ws(int T, int N, int K) {
    GemmArgs g{};
    g.E = 1;
    g.R = T;
    BackwardWs b{};
    b.dz = 0;
    b.db = up256((size_t)T * part_cols(N) * 2 * 2);
    b.gemm = b.db + up256((size_t)act_backward_slices(T, N) * N * 4);
    g.M = N;
    g.N = K;
    g.K = N;
    size_t n = 0;
    for (int64_t low : {(int64_t)0, part_cols(N)}) {
        g.a_low = low;
        n = std::max(n, std::max(gemm_ws_bytes(kGradRows, g), gemm_ws_bytes(kGradWeights, g)));
    }
    b.bytes = b.gemm + n;
    return b;
}

int check_act(int act) { return act < BITMOE_ACT_NONE || act > BITMOE_ACT_SILU ? BITMOE_EINVAL : BITMOE_OK; }

}  // namespace

extern "C" {

size_t moe_expert_matmul_workspace_bytes(int op, int E, int R, int N, int K) {
    if (check_sizes(E, R, N, K)) return 0;
    GemmArgs g{};
    g.E = E;
    g.R = R;
    switch (op) {
        case BITMOE_MATMUL: g.N = N; g.K = K; return gemm_ws_bytes(kForward, g);
        case BITMOE_MATMUL_DX: g.N = K; g.K = N; return gemm_ws_bytes(kGradRows, g);
        case BITMOE_MATMUL_DW: g.M = N; g.N = K; return gemm_ws_bytes(kGradWeights, g);
    }
    return 0;
}

int moe_expert_matmul(const bitmoe_rows *x, const bitmoe_experts *w, const int32_t *offsets, int R,
                      const bitmoe_rows *y, void *ws, size_t ws_bytes, void *stream) {
    return expert_rows_product(x, w, offsets, R, y, ws, ws_bytes, stream, false);
}

int moe_expert_matmul_dx(const bitmoe_rows *dy, const bitmoe_experts *w, const int32_t *offsets, int R,
                         const bitmoe_rows *dx, void *ws, size_t ws_bytes, void *stream) {
    return expert_rows_product(dy, w, offsets, R, dx, ws, ws_bytes, stream, true);
}

int moe_expert_matmul_dw(const bitmoe_rows *dy, const bitmoe_rows *x, const int32_t *offsets, int R,
                         const bitmoe_experts *dw, int accumulate, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_experts(dw, R);
    if (rc) return rc;
    if ((rc = check_rows(dy, R, dw->N, true)) || (rc = check_rows(x, R, dw->K, true))) return rc;
    if (!is16(dy->dtype) || x->dtype != dy->dtype || !out_type(dw->dtype, dy->dtype)) return BITMOE_EINVAL;
    if (!offsets || !aligned(offsets, 4)) return BITMOE_EINVAL;
    const GemmArgs g = weights_product(dy, x, offsets, R, dw, accumulate);
    if ((rc = check_ws(ws, ws_bytes, gemm_ws_bytes(kGradWeights, g)))) return rc;
    return launch_gemm(kGradWeights, dy->dtype, g, ws, as_stream(stream));
}

size_t moe_linear_workspace_bytes(int T, int N, int K) {
    if (check_sizes(1, T, N, K)) return 0;
    GemmArgs g{};
    g.E = 1;
    g.R = T;
    g.N = N;
    g.K = K;
    return gemm_ws_bytes(kForward, g);
}

int moe_linear(const bitmoe_rows *x, const bitmoe_experts *w, const void *bias, int act, const bitmoe_rows *residual,
               const bitmoe_rows *pre, const bitmoe_rows *y, void *ws, size_t ws_bytes, void *stream) {
    if (!x) return BITMOE_EINVAL;
    const int T = x->rows;
    int rc = check_experts(w, T);
    if (rc) return rc;
    if (w->E != 1 || (rc = check_act(act))) return BITMOE_EINVAL;
    if ((rc = check_rows(x, T, w->K, false)) || (rc = check_rows(y, T, w->N, false))) return rc;
    if (!is16(w->dtype) || x->dtype != w->dtype || !out_type(y->dtype, w->dtype)) return BITMOE_EINVAL;
    if (residual && ((rc = check_rows(residual, T, w->N, false)) || !out_type(residual->dtype, w->dtype)))
        return BITMOE_EINVAL;
    if (pre && ((rc = check_rows(pre, T, w->N, false)) || pre->dtype != w->dtype)) return BITMOE_EINVAL;
    if (bias && !aligned(bias, 2)) return BITMOE_EINVAL;
    if (T == 0) return BITMOE_OK;
    GemmArgs g = rows_product(x, w, nullptr, T, y, false);
    g.act = act;
    g.bias = bias;
    if (residual) {
        g.res = residual->data;
        g.ld_res = residual->ld;
        g.res_f32 = residual->dtype == BITMOE_F32;
    }
    if (pre) {
        g.pre = pre->data;
        g.ld_pre = pre->ld;
    }
    if ((rc = check_ws(ws, ws_bytes, gemm_ws_bytes(kForward, g)))) return rc;
    return launch_gemm(kForward, w->dtype, g, ws, as_stream(stream));
}

size_t moe_linear_backward_workspace_bytes(int T, int N, int K) {
    if (check_sizes(1, T, N, K)) return 0;
    return backward_ws(T, N, K).bytes;
}

int moe_linear_backward(const bitmoe_rows *dy, const bitmoe_rows *x, const bitmoe_experts *w, int act,
                        const bitmoe_rows *pre, const bitmoe_rows *dx, const bitmoe_experts *dw, void *db,
                        int db_dtype, void *ws, size_t ws_bytes, void *stream) {
    if (!dy) return BITMOE_EINVAL;
    const int T = dy->rows;
    int rc = check_experts(w, T);
    if (rc) return rc;
    const int N = w->N, K = w->K, dt = w->dtype;
    const bool rounded = act & BITMOE_ACT_ROUND_DZ;
    act &= ~BITMOE_ACT_ROUND_DZ;
    if (w->E != 1 || check_act(act) || !is16(dt)) return BITMOE_EINVAL;
    if ((rc = check_rows(dy, T, N, false)) || dy->dtype != dt) return BITMOE_EINVAL;
    if (act != BITMOE_ACT_NONE && ((rc = check_rows(pre, T, N, false)) || pre->dtype != dt)) return BITMOE_EINVAL;
    if (dx && ((rc = check_rows(dx, T, K, false)) || !out_type(dx->dtype, dt))) return BITMOE_EINVAL;
    if (dw) {
        if ((rc = check_rows(x, T, K, false)) || x->dtype != dt) return BITMOE_EINVAL;
        if ((rc = check_experts(dw, T))) return rc;
        if (dw->E != 1 || dw->N != N || dw->K != K || !out_type(dw->dtype, dt)) return BITMOE_EINVAL;
    }
    if (db && ((!is16(db_dtype) && db_dtype != BITMOE_F32) || !aligned(db, esize(db_dtype)))) return BITMOE_EINVAL;
    if (!dx && !dw && !db) return BITMOE_OK;
    const BackwardWs b = backward_ws(T, N, K);
    if ((rc = check_ws(ws, ws_bytes, b.bytes))) return rc;
    hipStream_t s = as_stream(stream);
    char *base = static_cast<char *>(ws);
    // dz replaces dy where there is an activation to differentiate (a launch of
    // its own: made inside the products it would be computed again by every
    // column's tiles, 28 times at K 7168): in two parts of the operands' type,
    // which double the products' time; in one where the caller takes that
    // rounding, or where it is none (relu)
    bitmoe_rows dz = *dy;
    const bool slope = act != BITMOE_ACT_NONE && (dx || dw);
    const int64_t low = slope && T > 0 && act != BITMOE_ACT_RELU && !rounded ? part_cols(N) : 0;
    if (slope && T > 0) {
        dz.data = base + b.dz;
        dz.ld = (low ? 2 : 1) * part_cols(N);
    }
    if (slope || db) {
        const ActBackward p{dy->data, act != BITMOE_ACT_NONE ? pre->data : nullptr, slope ? dz.data : nullptr,
                            dy->ld, act != BITMOE_ACT_NONE ? pre->ld : 0, dz.ld, low, T, N, act, db,
                            db_dtype, reinterpret_cast<float *>(base + b.db)};
        if ((rc = launch_act_backward(p, dt, s))) return rc;
    }
    if (dx && T > 0) {
        GemmArgs g = rows_product(&dz, w, nullptr, T, dx, true);
        g.a_low = low;
        if ((rc = launch_gemm(kGradRows, dt, g, base + b.gemm, s))) return rc;
    }
    if (dw) {
        GemmArgs g = weights_product(&dz, x, nullptr, T, dw, 0);
        g.a_low = low;
        if ((rc = launch_gemm(kGradWeights, dt, g, base + b.gemm, s))) return rc;
    }
    return BITMOE_OK;
}

int moe_swiglu(const bitmoe_rows *gate, const bitmoe_rows *up, const bitmoe_rows *h, void *stream) {
    if (!gate) return BITMOE_EINVAL;
    const int R = gate->rows, I = gate->cols, dt = gate->dtype;
    int rc = check_sizes(1, R, I, 1);
    if (rc) return rc;
    if (check_rows(gate, R, I, false) || check_rows(up, R, I, false) || check_rows(h, R, I, false))
        return BITMOE_EINVAL;
    if (!is16(dt) || up->dtype != dt || h->dtype != dt) return BITMOE_EINVAL;
    if (R == 0) return BITMOE_OK;
    return launch_swiglu(*gate, *up, *h, dt, as_stream(stream));
}

int moe_swiglu_backward(const bitmoe_rows *dh, const bitmoe_rows *gate, const bitmoe_rows *up,
                        const bitmoe_rows *dgate, const bitmoe_rows *dup, void *stream) {
    if (!gate) return BITMOE_EINVAL;
    const int R = gate->rows, I = gate->cols, dt = gate->dtype;
    int rc = check_sizes(1, R, I, 1);
    if (rc) return rc;
    for (const bitmoe_rows *m : {dh, gate, up, dgate, dup})
        if (check_rows(m, R, I, false) || m->dtype != dt) return BITMOE_EINVAL;
    if (!is16(dt)) return BITMOE_EINVAL;
    if (R == 0) return BITMOE_OK;
    return launch_swiglu_backward(*dh, *gate, *up, *dgate, *dup, dt, as_stream(stream));
}

int moe_combine(const bitmoe_rows *o, const float *w, int T, int k, const bitmoe_rows *residual,
                const bitmoe_rows *y, void *stream) {
    if (T < 0 || k < 1 || !o) return BITMOE_EINVAL;
    if (k > 16 || T > kMaxRows / k) return BITMOE_EUNSUPPORTED;
    const int H = o->cols;
    int rc = check_sizes(1, T, H, 1);
    if (rc) return rc;
    if (check_rows(o, T * k, H, false) || !is16(o->dtype)) return BITMOE_EINVAL;
    if (check_rows(y, T, H, false) || !out_type(y->dtype, o->dtype)) return BITMOE_EINVAL;
    if (residual && (check_rows(residual, T, H, false) || !out_type(residual->dtype, o->dtype))) return BITMOE_EINVAL;
    if (!aligned(w, 4)) return BITMOE_EINVAL;
    if (T == 0) return BITMOE_OK;
    return launch_combine(*o, w, T, k, residual, *y, as_stream(stream));
}

int moe_combine_backward(const bitmoe_rows *dy, const bitmoe_rows *o, const float *w, int T, int k,
                         const bitmoe_rows *d_o, float *dw, void *stream) {
    if (T < 0 || k < 1 || !dy || (!d_o && !dw) || (dw && !o)) return BITMOE_EINVAL;
    if (k > 16 || T > kMaxRows / k) return BITMOE_EUNSUPPORTED;
    const int H = dy->cols, dt = o ? o->dtype : d_o->dtype;
    int rc = check_sizes(1, T, H, 1);
    if (rc) return rc;
    if (!is16(dt) || check_rows(dy, T, H, false) || !out_type(dy->dtype, dt)) return BITMOE_EINVAL;
    if (o && (check_rows(o, T * k, H, false) || o->dtype != dt)) return BITMOE_EINVAL;
    if (d_o && (check_rows(d_o, T * k, H, false) || d_o->dtype != dt)) return BITMOE_EINVAL;
    if (!aligned(w, 4) || !aligned(dw, 4)) return BITMOE_EINVAL;
    if (T == 0) return BITMOE_OK;
    return launch_combine_backward(*dy, o, w, T, k, d_o, dw, dt, as_stream(stream));
}

}  // extern "C"
