"""Binding of the 16-bit expert layer and its gradients (bitmoe.h, "The layer
with 16-bit experts"): argument checks, output and workspace allocation, and
the call.

All operands are bfloat16 or float16 CUDA tensors of one type on one device,
with unit stride along their last dimension and any stride between rows.
Calls run on the current stream of the tensors' device, or on `stream` (of
that device), on which the outputs and workspaces they allocate then live;
inputs must be ready on it.  There is no autograd here: each gradient is a call
of its own.
"""
from __future__ import annotations

import struct

from ._lib import BF16, F16, F32, _check, _torch, lib

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
ROUND_DZ = 256          # or'ed to linear_backward's act
MATMUL, MATMUL_DX, MATMUL_DW = 0, 1, 2

# bitmoe_rows and bitmoe_experts as bytes: a call's operands are packed in a
# third of the time that ctypes structures take, which a small call feels
_ROWS = struct.Struct("@PPqiiii")
_EXPERTS = struct.Struct("@Pqqiiii")
_DTYPES = {}


def _dtype(t, what, f32=False):
    if not _DTYPES:
        torch = _torch()
        _DTYPES.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32})
    code = _DTYPES.get(t.dtype)
    if code is None or (code == F32 and not f32):
        raise TypeError(f"{what} must be bfloat16 or float16" + (" or float32" if f32 else ""))
    return code


def _strided(n, cols, stride, what):
    """Elements between the n rows of a matrix (the last two dimensions)."""
    if n == 0 or cols == 0:
        return cols
    ld, one = stride[-2:]
    if one != 1 and cols > 1:
        raise ValueError(f"{what} must have unit stride along its last dimension")
    if ld < cols:
        # (a single row has no stride of its own; rows that overlap, as an expanded tensor's do, are refused)
        if n > 1:
            raise ValueError(f"{what} must have rows that do not overlap")
        ld = cols
    return ld


def _rows(t, what, shape=None, rows_map=None, div=1, f32=False):
    """A bitmoe_rows; shape: what the call needs (None for any number of
    rows)."""
    at = t.shape
    if len(at) != 2:
        raise ValueError(f"{what} must have 2 dimensions")
    n, cols = at
    if shape is not None and (cols != shape[1] or (shape[0] is not None and n != shape[0])):
        raise ValueError(f"{what} must be [{'n' if shape[0] is None else shape[0]}, {shape[1]}]")
    ld, code = _strided(n, cols, t.stride(), what), _dtype(t, what, f32)
    try:
        return _ROWS.pack(t.data_ptr(), 0 if rows_map is None else rows_map.data_ptr(), ld, n, cols, div, code)
    except struct.error:
        raise ValueError(f"{what} or its map's divisor is too large") from None


def _experts(t, what, shape=None, f32=False):
    """A bitmoe_experts: [E, N, K], or [N, K] as a single expert's."""
    at, stride = t.shape, t.stride()
    if shape is not None and tuple(at) != shape:
        raise ValueError(f"{what} must be {list(shape)}")
    if len(at) == 2:
        (N, K), E = at, 1
    elif len(at) == 3:
        E, N, K = at
    else:
        raise ValueError(f"{what} must have 3 dimensions")
    ld = _strided(N, K, stride, what)
    return _EXPERTS.pack(t.data_ptr(), ld, stride[0] if E > 1 else N * ld, E, N, K, _dtype(t, what, f32))


def _ints(t, what, n=None):
    if t.dtype != _torch().int32 or t.dim() != 1 or (t.stride(0) != 1 and t.numel() > 1):
        raise ValueError(f"{what} must be a contiguous one-dimensional int32 tensor")
    if n is not None and t.numel() != n:
        raise ValueError(f"{what} must have {n} elements")
    return t.numel()


def _device(*ts):
    """The index of the tensors' one device."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must be on one device")
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    return dev


def _current_stream(dev):
    """The current stream's handle (without a torch.cuda.Stream object, where
    torch offers that: 1 us less per call)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _elsewhere(dev, stream):
    """None, or what makes a call run on `stream` (so that what it allocates
    lives there) or on another device than the current one."""
    torch = _torch()
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("the stream must be on the tensors' device")
        return torch.cuda.stream(stream)
    return None if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _output(t, shape, dtype, dev, what, wanted=None):
    """The given output, or a new one of dtype."""
    if t is None:
        return _torch().empty(shape, dtype=dtype, device=dev)
    if wanted is not None and t.dtype != wanted:
        raise ValueError(f"{what} is not of out_dtype")
    return t


def _scratch(ws, need, dev):
    """(the tensor, its address, its bytes)"""
    if ws is None:
        if not need:
            return None, None, 0
        torch = _torch()
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not ws.is_contiguous() or ws.dtype != _torch().uint8:
        raise ValueError("ws must be a contiguous uint8 tensor")
    return ws, ws.data_ptr(), ws.numel()


def expert_matmul_workspace_bytes(op: int, E: int, R: int, N: int, K: int) -> int:
    """Workspace of an expert product (op MATMUL, MATMUL_DX or MATMUL_DW) over
    R rows, experts of N x K."""
    return int(lib().moe_expert_matmul_workspace_bytes(op, E, R, N, K))


def _expert_rows(op, a, w, offsets, a_rows, a_div, c_rows, c, out_dtype, ws, stream):
    dev = _device(a, w, offsets, a_rows, c_rows, c, ws)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return _expert_rows(op, a, w, offsets, a_rows, a_div, c_rows, c, out_dtype, ws, None)
    an, cn = ("x", "y") if op == MATMUL else ("dy", "dx")
    if len(w.shape) != 3:
        raise ValueError("w must have 3 dimensions")
    we = _experts(w, "w")
    E, N, K = w.shape
    n_in, n_out = (K, N) if op == MATMUL else (N, K)
    R = _ints(a_rows, f"{an}_rows") if a_rows is not None else None
    if c_rows is not None:
        n = _ints(c_rows, f"{cn}_rows")
        if R is None:
            R = n
            if n > a.shape[0]:
                raise ValueError(f"{cn}_rows must not be longer than {an}")
        elif n != R:
            raise ValueError(f"{an}_rows and {cn}_rows must have the same length")
    elif R is None:
        R = a.shape[0]
    _ints(offsets, "offsets", E + 1)
    ar = _rows(a, an, (None, n_in), a_rows, a_div)
    if a.dtype != w.dtype:
        raise ValueError(f"{an} must be of w's type")
    ungrouped = c is None and c_rows is not None
    c = _output(c, (R, n_out), out_dtype or a.dtype, dev, cn, out_dtype)
    cr = _rows(c, cn, (None, n_out), c_rows, 1, f32=True)
    L = lib()
    hold, p, n = _scratch(ws, L.moe_expert_matmul_workspace_bytes(op, E, R, N, K), dev)
    s = _current_stream(dev)
    if ungrouped:
        _check(L.moe_expert_clear_ungrouped(offsets.data_ptr(), E, R, cr, s), "moe_expert_clear_ungrouped")
    if op == MATMUL:
        _check(L.moe_expert_matmul(ar, we, offsets.data_ptr(), R, cr, p, n, s), "moe_expert_matmul")
    else:
        _check(L.moe_expert_matmul_dx(ar, we, offsets.data_ptr(), R, cr, p, n, s), "moe_expert_matmul_dx")
    return c


def expert_matmul(x, w, offsets, x_rows=None, x_div=1, y_rows=None, y=None, out_dtype=None, ws=None, stream=None):
    """y[r] = W_e x[r] for the rows r of expert e, offsets[e] <= r < offsets[e+1].

    x [n, K], w [E, N, K], offsets int32 [E + 1] (bucket's).  x_rows int32 [R]:
    row r is x[x_rows[r] // x_div] (bucket's perm with x_div = k gathers each
    pair's token); y_rows int32 [R]: row r goes to y[y_rows[r]] (perm: pair
    order).  Without them row r is row r.  An entry outside the matrix reads as
    zeros, or is not written.  Returns y [R, N] in out_dtype (default x's;
    float32 allowed).  Rows of y that no group's row is written to are left as
    they were.  Where this call allocates y and y_rows is given, those that the
    rows of no group go to are 0 (over a share of the experts, the other shares'
    pairs: w[e0:e1], offsets[e0:e1 + 1]); without y_rows they are undefined."""
    return _expert_rows(MATMUL, x, w, offsets, x_rows, x_div, y_rows, y, out_dtype, ws, stream)


def expert_matmul_dx(dy, w, offsets, dy_rows=None, dy_div=1, dx_rows=None, dx=None, out_dtype=None, ws=None,
                     stream=None):
    """dx[r] = W_e^T dy[r], the gradient of expert_matmul's x for each of the
    R rows (dy [n, N] -> dx [R, K]); maps as in expert_matmul."""
    return _expert_rows(MATMUL_DX, dy, w, offsets, dy_rows, dy_div, dx_rows, dx, out_dtype, ws, stream)


def expert_matmul_dw(dy, x, offsets, dy_rows=None, dy_div=1, x_rows=None, x_div=1, dw=None, out_dtype=None,
                     accumulate=False, ws=None, stream=None):
    """dW_e = sum over e's rows r of dy[r] x[r]^T, the gradient of
    expert_matmul's w: dw [E, N, K] (0 for an expert without rows; added to
    what dw holds if accumulate); maps as in expert_matmul."""
    dev = _device(dy, x, offsets, dy_rows, x_rows, dw, ws)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return expert_matmul_dw(dy, x, offsets, dy_rows, dy_div, x_rows, x_div, dw, out_dtype, accumulate, ws)
    R = dy.shape[0] if dy_rows is None else _ints(dy_rows, "dy_rows")
    if R != (x.shape[0] if x_rows is None else _ints(x_rows, "x_rows")):
        raise ValueError("dy and x must give the same number of rows")
    if dy.dtype != x.dtype:
        raise ValueError("dy and x must be of one type")
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    E = _ints(offsets, "offsets") - 1
    dr, xr = _rows(dy, "dy", None, dy_rows, dy_div), _rows(x, "x", None, x_rows, x_div)
    N, K = dy.shape[1], x.shape[1]
    dw = _output(dw, (E, N, K), out_dtype or x.dtype, dev, "dw", out_dtype)
    d = _experts(dw, "dw", (E, N, K), f32=True)
    L = lib()
    hold, p, n = _scratch(ws, L.moe_expert_matmul_workspace_bytes(MATMUL_DW, E, R, N, K), dev)
    _check(L.moe_expert_matmul_dw(dr, xr, offsets.data_ptr(), R, d, 1 if accumulate else 0, p, n,
                                  _current_stream(dev)), "moe_expert_matmul_dw")
    return dw


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}")
    return ACTS[act]


def _vector(t, n, what):
    if tuple(t.shape) != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous tensor of {n} values")
    return t.data_ptr()


def linear(x, w, bias=None, act="none", residual=None, keep_pre=False, y=None, pre=None, out_dtype=None, ws=None,
           stream=None):
    """y = act(x w^T + bias) + residual.  x [T, K], w [N, K], bias [N],
    residual [T, N] (x's type or float32); act: a key of ACTS.  Returns
    (y, pre): y [T, N] in out_dtype (default x's), pre the value before act (x's
    type, for linear_backward) if keep_pre or given, else None.  y may be the
    residual itself."""
    code = _act(act)
    dev = _device(x, w, bias, residual, y, pre, ws)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return linear(x, w, bias, act, residual, keep_pre, y, pre, out_dtype, ws)
    if len(w.shape) != 2:
        raise ValueError("w must have 2 dimensions")
    we = _experts(w, "w")
    N, K = w.shape
    xr = _rows(x, "x", (None, K))
    dtype, T = x.dtype, x.shape[0]
    if dtype != w.dtype or (bias is not None and bias.dtype != dtype):
        raise ValueError("x, w and bias must be of one type")
    shape = (T, N)
    b = None if bias is None else _vector(bias, N, "bias")
    rr = None if residual is None else _rows(residual, "residual", shape, f32=True)
    y = _output(y, shape, out_dtype or dtype, dev, "y", out_dtype)
    yr = _rows(y, "y", shape, f32=True)
    if pre is None and keep_pre:
        pre = _torch().empty(shape, dtype=dtype, device=dev)
    pr = None if pre is None else _rows(pre, "pre", shape)
    L = lib()
    hold, p, n = _scratch(ws, L.moe_linear_workspace_bytes(T, N, K), dev)
    _check(L.moe_linear(xr, we, b, code, rr, pr, yr, p, n, _current_stream(dev)), "moe_linear")
    return y, pre


def linear_backward(dy, x, w, act="none", pre=None, dx=None, dw=None, db=None, need_dx=True, need_dw=True,
                    need_db=False, out_dtype=None, ws=None, stream=None, round_dz=False):
    """Gradients of linear: with dz = dy act'(pre), (dx, dw, db) = (dz w,
    dz^T x, column sums of dz), None for what is not needed (given outputs are
    needed); new ones in out_dtype (default x's).  The residual's gradient is
    dy.  round_dz: dz is rounded to x's type before the products, which then
    take half their time (else it enters them as two such values; db sums dz
    itself either way)."""
    code = _act(act)
    if code and pre is None:
        raise ValueError("pre is needed with an activation")
    dev = _device(dy, x, w, pre, dx, dw, db, ws)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return linear_backward(dy, x, w, act, pre, dx, dw, db, need_dx, need_dw, need_db, out_dtype, ws,
                                   round_dz=round_dz)
    if len(w.shape) != 2:
        raise ValueError("w must have 2 dimensions")
    we = _experts(w, "w")
    N, K = w.shape
    T, dtype = dy.shape[0], w.dtype
    if x.dtype != dtype or dy.dtype != dtype or (code and pre.dtype != dtype):
        raise ValueError("dy, x and pre must be of w's type")
    dyr, xr = _rows(dy, "dy", (None, N)), _rows(x, "x", (T, K))
    pr = _rows(pre, "pre", (T, N)) if code else None
    new = out_dtype or dtype
    dx = _output(dx, (T, K), new, dev, "dx") if dx is not None or need_dx else None
    dw = _output(dw, (N, K), new, dev, "dw") if dw is not None or need_dw else None
    db = _output(db, (N,), new, dev, "db") if db is not None or need_db else None
    dxr = None if dx is None else _rows(dx, "dx", (T, K), f32=True)
    dwe = None if dw is None else _experts(dw, "dw", (N, K), f32=True)
    dbp, dbt = (None, F32) if db is None else (_vector(db, N, "db"), _dtype(db, "db", True))
    L = lib()
    hold, p, n = _scratch(ws, L.moe_linear_backward_workspace_bytes(T, N, K), dev)
    _check(L.moe_linear_backward(dyr, xr, we, code | (ROUND_DZ if round_dz else 0), pr, dxr, dwe, dbp, dbt, p, n,
                                 _current_stream(dev)), "moe_linear_backward")
    return dx, dw, db


def _one_type(names, first, *ts):
    for t in ts:
        if t.dtype != first.dtype:
            raise ValueError(f"{names} must be of one type")


def swiglu(gate, up, h=None, stream=None):
    """h = silu(gate) * up, all [R, I] with any row stride (gate and up may be
    the halves of one product's output).  h may be gate or up."""
    dev = _device(gate, up, h)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return swiglu(gate, up, h)
    shape = gate.shape
    g = _rows(gate, "gate")
    h = _output(h, shape, gate.dtype, dev, "h")
    _one_type("gate, up and h", gate, up, h)
    _check(lib().moe_swiglu(g, _rows(up, "up", shape), _rows(h, "h", shape), _current_stream(dev)), "moe_swiglu")
    return h


def swiglu_backward(dh, gate, up, dgate=None, dup=None, stream=None):
    """Gradients of swiglu: (dgate, dup).  Without them given, both are views
    of one new [R, 2 I] matrix, gate's half first."""
    dev = _device(dh, gate, up, dgate, dup)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return swiglu_backward(dh, gate, up, dgate, dup)
    if (dgate is None) != (dup is None):
        raise ValueError("dgate and dup are given together")
    shape = gate.shape
    g = _rows(gate, "gate")
    if dgate is None:
        both = _torch().empty((shape[0], 2 * shape[1]), dtype=gate.dtype, device=dev)
        dgate, dup = both[:, :shape[1]], both[:, shape[1]:]
    _one_type("dh, gate, up, dgate and dup", gate, dh, up, dgate, dup)
    _check(lib().moe_swiglu_backward(_rows(dh, "dh", shape), g, _rows(up, "up", shape), _rows(dgate, "dgate", shape),
                                     _rows(dup, "dup", shape), _current_stream(dev)), "moe_swiglu_backward")
    return dgate, dup


def _weights(w, k, n, what):
    """(T, k, the weights' address) of a combine over n expert rows."""
    if w is not None:
        if w.dim() != 2 or w.dtype != _torch().float32 or not w.is_contiguous():
            raise ValueError("w must be a contiguous float32 [T, k]")
        T, wk = w.shape
        if k is not None and k != wk:
            raise ValueError("k is not w's")
        if T * wk != n:
            raise ValueError(f"{what} must have T * k rows")
        return T, wk, w.data_ptr()
    if k is None or k < 1 or n % k:
        raise ValueError(f"without w, k is needed and {what} has T * k rows")
    return n // k, k, None


def combine(o, w=None, k=None, residual=None, y=None, out_dtype=None, stream=None):
    """y[t] = sum_j w[t, j] o[t k + j] + residual[t].  o [T k, H], w float32
    [T, k] (None: ones, with k given), residual [T, H] (o's type or float32).
    y [T, H] in out_dtype (default the residual's, else o's; o's or float32); y
    may be the residual itself."""
    dev = _device(o, w, residual, y)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return combine(o, w, k, residual, y, out_dtype)
    orow = _rows(o, "o")
    T, k, wp = _weights(w, k, o.shape[0], "o")
    shape = (T, o.shape[1])
    rr = None if residual is None else _rows(residual, "residual", shape, f32=True)
    y = _output(y, shape, out_dtype or (o if residual is None else residual).dtype, dev, "y", out_dtype)
    _check(lib().moe_combine(orow, wp, T, k, rr, _rows(y, "y", shape, f32=True), _current_stream(dev)), "moe_combine")
    return y


def combine_backward(dy, o=None, w=None, k=None, d_o=None, dw=None, need_do=True, need_dw=True, stream=None):
    """Gradients of combine: (d_o, dw) with d_o[t k + j] = w[t, j] dy[t] (o's
    type) and dw[t, j] = <dy[t], o[t k + j]> (float32); None for one not
    needed.  Without o (then need_dw = False) d_o is of dy's type.  The
    residual's gradient is dy.  d_o may be o itself."""
    need_dw = need_dw or dw is not None
    need_do = need_do or d_o is not None
    if need_dw and o is None:
        raise ValueError("dw needs o")
    if o is None and w is None and k is None:
        raise ValueError("without o and w, k is needed")
    dev = _device(dy, o, w, d_o, dw)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return combine_backward(dy, o, w, k, d_o, dw, need_do, need_dw)
    T, k, wp = _weights(w, k, o.shape[0] if o is not None else dy.shape[0] * (w.shape[1] if w is not None else k), "o")
    yr = _rows(dy, "dy", (T, dy.shape[-1]), f32=True)
    shape = (T * k, dy.shape[1])
    orow = None if o is None else _rows(o, "o", shape)
    if not need_do and not need_dw:
        return None, None
    dr = dp = None
    if need_do:
        d_o = _output(d_o, shape, (dy if o is None else o).dtype, dev, "d_o")
        dr = _rows(d_o, "d_o", shape)
    if need_dw:
        torch = _torch()
        dw = _output(dw, (T, k), torch.float32, dev, "dw", torch.float32)
        if tuple(dw.shape) != (T, k) or not dw.is_contiguous():
            raise ValueError(f"dw must be a contiguous float32 [{T}, {k}]")
        dp = dw.data_ptr()
    _check(lib().moe_combine_backward(yr, orow, wp, T, k, dr, dp, _current_stream(dev)), "moe_combine_backward")
    return d_o, dw
