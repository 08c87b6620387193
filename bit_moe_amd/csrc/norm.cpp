// C ABI of the norms around a block: host-side validation, as in experts.cpp
// (every check runs before the first launch).
#include "norm.h"

namespace {

using namespace bm_host;

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

NormMat mat(const bitmoe_rows *m) { return m ? NormMat{m->data, m->ld, m->dtype == BITMOE_F32} : NormMat{nullptr, 0, false}; }

// the call's tokens, columns and 16-bit type, from the first operands that are there
struct Call {
    int T, H, dt;
};
int check_call(const bitmoe_rows *sized, const bitmoe_rows *typed, Call *c) {
    if (!sized || !typed || !is16(typed->dtype)) return BITMOE_EINVAL;
    *c = Call{sized->rows, sized->cols, typed->dtype};
    const int rc = check_sizes(1, c->T, c->H, 1);
    if (rc) return rc;
    return c->H > kMaxNormCols ? BITMOE_EUNSUPPORTED : BITMOE_OK;
}
// m: not there, or the call's rows of its 16-bit type (or, with f32, float32)
bool fits(const bitmoe_rows *m, const Call &c, bool f32) {
    return !m || (!check_rows(m, c.T, c.H, false) && (f32 ? out_type(m->dtype, c.dt) : m->dtype == c.dt));
}
// a gate of the call's rows, or of one row for all
bool gate_fits(const bitmoe_rows *m, const Call &c, bool *one) {
    *one = m && m->rows == 1;
    return *one ? !check_rows(m, 1, c.H, false) && m->dtype == c.dt : fits(m, c, false);
}
bool eps_ok(float eps) { return eps >= kMinEps && eps <= 3.4028234e38f; }

}  // namespace

extern "C" {

int moe_block_norm(const bitmoe_rows *o, const void *w_after, const bitmoe_rows *gate, const bitmoe_rows *residual,
                   float scale, const bitmoe_rows *s, const void *w_before, float eps, const bitmoe_rows *n,
                   void *stream) {
    Call c;
    const int rc = check_call(o ? o : residual, o ? o : n, &c);
    if (rc) return rc;
    bool one;
    if (!fits(o, c, false) || !fits(residual, c, true) || !fits(s, c, true) || !fits(n, c, false)) return BITMOE_EINVAL;
    if (!gate_fits(gate, c, &one) || (!o && (gate || w_after)) || (!s && !n)) return BITMOE_EINVAL;
    if (!aligned(w_after, 2) || !aligned(w_before, 2) || !eps_ok(eps)) return BITMOE_EINVAL;
    if (c.T == 0) return BITMOE_OK;
    NormArgs a{};
    a.o = mat(o);
    a.gate = mat(gate);
    if (one) a.gate.ld = 0;
    a.res = mat(residual);
    a.s = mat(s);
    a.n = mat(n);
    a.wa = w_after;
    a.wb = w_before;
    a.scale = scale;
    a.eps = eps;
    a.T = c.T;
    a.H = c.H;
    return launch_block_norm(a, c.dt, as_stream(stream));
}

size_t moe_block_norm_backward_workspace_bytes(int T, int H) {
    if (check_sizes(1, T, H, 1) || H > kMaxNormCols) return 0;
    return up256((size_t)norm_shape(T, H).slices * 2 * H * 4);
}

int moe_block_norm_backward(const bitmoe_rows *dn, const bitmoe_rows *ds, const bitmoe_rows *s, const bitmoe_rows *o,
                            const void *w_after, const bitmoe_rows *gate, float scale, const void *w_before,
                            float eps, const bitmoe_rows *d_o, const bitmoe_rows *dresidual, void *dw_after,
                            const bitmoe_rows *dgate, void *dw_before, int dw_dtype, void *ws, size_t ws_bytes,
                            void *stream) {
    Call c;
    const int rc = check_call(dn ? dn : ds, dn ? dn : o, &c);
    if (rc) return rc;
    bool one;
    for (const bitmoe_rows *m : {dn, o, d_o})
        if (!fits(m, c, false)) return BITMOE_EINVAL;
    for (const bitmoe_rows *m : {ds, s, dresidual})
        if (!fits(m, c, true)) return BITMOE_EINVAL;
    if (!gate_fits(gate, c, &one) || !aligned(w_after, 2) || !aligned(w_before, 2) || !eps_ok(eps)) return BITMOE_EINVAL;
    if ((dn && !s) || (!dn && (dw_before || w_before)) || (!o && (gate || w_after || d_o || dw_after))) return BITMOE_EINVAL;
    if (dw_dtype != c.dt && dw_dtype != BITMOE_F32) return BITMOE_EINVAL;
    for (const void *p : {(const void *)dw_after, (const void *)dw_before})
        if (!aligned(p, esize(dw_dtype))) return BITMOE_EINVAL;
    if (dgate && !gate) return BITMOE_EINVAL;
    if (one && dgate) {
        if (check_rows(dgate, 1, c.H, false) || !out_type(dgate->dtype, c.dt)) return BITMOE_EINVAL;
    } else if (!fits(dgate, c, false)) {
        return BITMOE_EINVAL;
    }
    if (!d_o && !dresidual && !dw_after && !dgate && !dw_before) return BITMOE_OK;
    const size_t need = moe_block_norm_backward_workspace_bytes(c.T, c.H);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return BITMOE_EWORKSPACE;
    NormBackArgs a{};
    a.dn = mat(dn);
    a.ds = mat(ds);
    a.s = mat(dn ? s : nullptr);
    a.o = mat(o);
    a.gate = mat(gate);
    if (one) a.gate.ld = 0;
    a.d_o = mat(d_o);
    a.dres = mat(dresidual);
    a.dgate = mat(one ? nullptr : dgate);
    a.wa = w_after;
    a.wb = w_before;
    a.scale = scale;
    a.eps = eps;
    a.T = c.T;
    a.H = c.H;
    a.dwa = dw_after;
    a.dwb = dw_before;
    a.dg = one && dgate ? dgate->data : nullptr;
    a.dw_dtype = dw_dtype;
    a.dg_dtype = one && dgate ? dgate->dtype : dw_dtype;
    a.partial = static_cast<float *>(ws);
    return launch_block_norm_backward(a, c.dt, as_stream(stream));
}

}  // extern "C"
