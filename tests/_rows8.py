"""The expert layer's operators in 8 bits and the norms around a block by their
formulas, in float64 on the CPU (the tests' oracle), and bounds on what the
kernels' arithmetic may differ from them by."""
import torch

import _experts as ex

F64 = ex.F64
U = 2.0 ** -24                # half a step of float32


def blocks_of(x, block):
    """x [R, C] as [R, blocks, columns of one], zeros behind the last column."""
    b = block or x.shape[1]
    return torch.nn.functional.pad(x, (0, -x.shape[1] % b)).view(x.shape[0], -1, b)


def quantize(x, block=0):
    """(quotients 127 x / m, codes, scales [R, blocks]) of rows in 8 bits."""
    v = blocks_of(x, block)
    m = v.abs().amax(2, keepdim=True)
    t = torch.where(m > 0, 127 * v / m, torch.zeros_like(v)).reshape(x.shape[0], -1)[:, :x.shape[1]]
    return t, t.round(), m[:, :, 0] / 127


def values(codes, scale, block=0):
    """codes * scale, both float64; scale [R] (block 0) or [R, blocks]."""
    if not block:
        return codes * scale[:, None]
    return codes * scale.repeat_interleave(block, 1)[:, :codes.shape[1]]


def silu_bound(g):
    """Relative error of the kernels' silu(g): e^-g by 2^(g log2 e) has |g| 2^-24
    from its argument and a step of its own, then a sum, a quotient and products."""
    return (g.abs() + 8) * 2 * U


def slope_bound(dh, g, u):
    """Error of dh u p (1 + g (1 - p)): the bracket's terms may cancel, so against
    their absolute values; p's relative error as silu's, twice."""
    p = torch.sigmoid(g)
    return (dh * u).abs() * p * (1 + g.abs()) * (g.abs() + 16) * 2 * U


def expert_rows(codes, scale, w, w_scale, offsets):
    """y[r] = (sum of the codes' products) * scale[r] * w_scale[e][n] by groups of
    rows, all float64 (the sums are exact: below 2^31)."""
    y = torch.zeros(codes.shape[0], w.shape[1], dtype=F64)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        y[s] = codes[s] @ w[e].t() * scale[s, None] * w_scale[e][None]
    return y


def product_bound(want, dtype):
    """The sum to float32, two products and the rounding to the output's type
    (float16's smallest values are half a step of 2^-24 off)."""
    return (ex.half_ulp(dtype) * (1 + 4 * U) + 3.01 * U) * want.abs() + 2.0 ** -25 * (dtype == torch.float16)


# ---- norms ----------------------------------------------------------------

def unit(v, eps):
    """v / rms(v), 1 / rms(v)."""
    inv = (v.square().mean(1, keepdim=True) + eps) ** -0.5
    return v * inv, inv


def block_norm(o, residual, wa, gate, scale, wb, eps):
    s = 0 if residual is None else scale * residual
    if o is not None:
        s = s + gate * unit(o, eps)[0] * wa
    return s, unit(s, eps)[0] * wb


def block_norm_backward(dn, ds, s, o, wa, gate, scale, wb, eps):
    """(d_o, dresidual, dw_after, dgate by token, dw_before by token's sum), by the
    formulas."""
    H = (ds if dn is None else dn).shape[1]
    t = torch.zeros_like(dn) if ds is None else ds
    dwb = None
    if dn is not None:
        sn, b = unit(s, eps)
        p = dn * wb
        t = t + b * (p - sn * (p * sn).sum(1, keepdim=True) / H)
        dwb = (dn * sn).sum(0)
    if o is None:
        return None, scale * t, None, None, dwb
    on, a = unit(o, eps)
    v = gate * t * wa
    return a * (v - on * (v * on).sum(1, keepdim=True) / H), scale * t, (gate * t * on).sum(0), t * on * wa, dwb


# Every thread adds at most 16 squares in turn, 64 lanes meet in 6 steps and 16
# waves in 15: a value passes at most 37 additions, and one fma's rounding.  With
# the division, eps, and the root's own step 1 / rms is within 19 + 3 steps, taken
# as 24; a normed value has 4 more products, taken as 32 in all.
INV, NORMED, SUM = 24 * U, 32 * U, 40 * U


def norm_bounds(o, residual, wa, gate, scale, wb, eps, s_dtype, n_dtype):
    """Bounds of s and n."""
    s, n = block_norm(o, residual, wa, gate, scale, wb, eps)
    e = 0 if residual is None else 2 * U * (scale * residual).abs()
    if o is not None:
        e = e + NORMED * (gate * unit(o, eps)[0] * wa).abs()
    e = e + U * s.abs()
    inv = unit(s, eps)[1]
    small = lambda d: 2.0 ** -25 * (d == torch.float16)  # noqa: E731
    es = ex.half_ulp(s_dtype) * s.abs() * (1 + U) + e + small(s_dtype)
    # the errors of s in s itself and, by its length, in 1 / rms
    en = e * inv * wb.abs() + n.abs() * (NORMED + e.square().mean(1, keepdim=True).sqrt() * inv)
    return s, n, es, ex.half_ulp(n_dtype) * n.abs() + en + small(n_dtype)


def norm_backward_bounds(dn, ds, s, o, wa, gate, scale, wb, eps, dtype, dres_dtype, dw_dtype):
    """(values, bounds) of d_o, dresidual, dw_after, dgate (by token; and summed),
    dw_before: each term's own rounding, and the sums' against their absolute
    values, as <v, o> is taken in three sums whose parts may cancel."""
    first = ds if dn is None else dn
    T, H = first.shape
    d_o, dres, dwa, dg, dwb = block_norm_backward(dn, ds, s, o, wa, gate, scale, wb, eps)
    t = dres / scale
    zero = torch.zeros_like(first)
    parts = zero if ds is None else ds.abs()
    et = 2 * U * parts
    bounds = {}
    small = lambda d: 2.0 ** -25 * (d == torch.float16)  # noqa: E731
    tokens = ex.sum_bound(T)
    if dn is not None:
        sn, b = unit(s, eps)
        p = (dn * wb).abs()
        mean = (p * sn.abs()).sum(1, keepdim=True) / H
        et = et + b * (p * (INV + 4 * U) + sn.abs() * mean * (SUM + 2 * INV + 8 * U))
        parts = parts + b * (p + sn.abs() * mean)
        bounds["dw_before"] = (dn * sn).abs().sum(0) * (INV + 2 * U + tokens) + ex.half_ulp(dw_dtype) * dwb.abs() + small(dw_dtype)
    et = et + U * t.abs()
    bounds["dresidual"] = abs(scale) * et + (ex.half_ulp(dres_dtype) + 2 * U) * dres.abs() + small(dres_dtype)
    if o is not None:
        on, a = unit(o, eps)
        gw = (gate * wa).abs()
        vo = (gw * on.abs() * parts).sum(1, keepdim=True) / H
        e = gw * (et + t.abs() * 8 * U) + on.abs() * vo * (SUM + 2 * INV + 2 * INV + 12 * U)
        bounds["d_o"] = a * (e + (gw * t.abs() + on.abs() * vo) * (INV + 4 * U)) + ex.half_ulp(dtype) * d_o.abs() + small(dtype)
        term = on.abs() * (et + t.abs() * (INV + 8 * U))
        eg = term * wa.abs()
        bounds["dgate"] = eg + ex.half_ulp(dtype) * dg.abs() + small(dtype)
        bounds["dgate_sum"] = eg.sum(0) + tokens * dg.abs().sum(0) + ex.half_ulp(dw_dtype) * dg.sum(0).abs() + small(dw_dtype)
        bounds["dw_after"] = ((term * gate.abs()).sum(0) + tokens * (gate * t * on).abs().sum(0) +
                              ex.half_ulp(dw_dtype) * dwa.abs() + small(dw_dtype))
    return {"d_o": d_o, "dresidual": dres, "dw_after": dwa, "dgate": dg,
            "dgate_sum": None if dg is None else dg.sum(0), "dw_before": dwb}, bounds
