"""The 16-bit expert layer's operators by their formulas, in float64 on the
CPU (the tests' oracle), and bounds on what the kernels' arithmetic may differ
from them by."""
import math

import torch

F64 = torch.float64


def half_ulp(dtype):
    """The largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


def sum_bound(n):
    """A sum of n products in fp32, in any order: n roundings of partial sums,
    each at most 2^-24 of the absolute values' sum, twice that for a matrix
    core's inner sums, whose roundings need not be to nearest."""
    return 2 * (n + 2) * 2.0 ** -24


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def mapped(a, rows, div=1):
    """The call's rows of matrix a; zeros where the map gives none."""
    if rows is None:
        return a
    at = torch.div(rows.long(), div, rounding_mode="floor")
    ok = (rows >= 0) & (at < a.shape[0])
    out = torch.zeros(rows.numel(), a.shape[1], dtype=a.dtype)
    out[ok] = a[at[ok]]
    return out


def expert_rows(x, w, offsets, transposed=False):
    """y[r] = W_e x[r] (W_e^T x[r]) and the sum of the products' absolute
    values; rows of no group are zero."""
    y = torch.zeros(x.shape[0], w.shape[2 if transposed else 1], dtype=F64)
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        m = w[e] if transposed else w[e].t()
        y[s] = x[s] @ m
        mag[s] = x[s].abs() @ m.abs()
    return y, mag


def expert_dw(dy, x, offsets):
    E = offsets.numel() - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=F64)
    mag = torch.zeros_like(dw)
    for e in range(E):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        dw[e] = dy[s].t() @ x[s]
        mag[e] = dy[s].abs().t() @ x[s].abs()
    return dw, mag


def swiglu(g, u):
    return act(g, "silu") * u


def swiglu_backward(dh, g, u):
    return dh * u * act_slope(g, "silu"), dh * act(g, "silu")


def combine(o, w, T, k, residual=None):
    y = (o.view(T, k, -1) * w[:, :, None]).sum(1)
    return y if residual is None else y + residual


def combine_backward(dy, o, w, T, k):
    return ((w[:, :, None] * dy[:, None, :]).reshape(T * k, -1), (o.view(T, k, -1) * dy[:, None, :]).sum(2))
