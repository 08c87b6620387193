"""Binding of the 16-bit expert layer and its gradients (bitmoe.h, "The layer
with 16-bit experts"): argument checks, output and workspace allocation, and
the call.

All operands are bfloat16 or float16 CUDA tensors of one type on one device,
with unit stride along their last dimension and any stride between rows.
Calls run on the current stream of the tensors' device, or on `stream` (of
that device), on which the outputs and workspaces they allocate then live;
inputs must be ready on it.  There is no autograd here: each gradient is a call of its own.
"""
from __future__ import annotations

import ctypes as C

from ._lib import BF16, F16, F32, ExpertsStruct, RowsStruct, _check, _torch, lib

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
MATMUL, MATMUL_DX, MATMUL_DW = 0, 1, 2


def _codes():
    torch = _torch()
    return {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}


_DTYPES = None


def _dtype(t, what, f32=False):
    global _DTYPES
    if _DTYPES is None:
        _DTYPES = _codes()
    code = _DTYPES.get(t.dtype)
    if code is None or (code == F32 and not f32):
        raise TypeError(f"{what} must be bfloat16 or float16" + (" or float32" if f32 else ""))
    return code


def _strided(shape, stride, what):
    """Elements between rows of a matrix (the last two dimensions)."""
    n, cols = shape[-2], shape[-1]
    if n == 0 or cols == 0:
        return cols
    if cols > 1 and stride[-1] != 1:
        raise ValueError(f"{what} must have unit stride along its last dimension")
    ld = stride[-2]
    if ld < cols:
        # (a single row has no stride of its own; rows that overlap, as an expanded tensor's do, are refused)
        if n > 1:
            raise ValueError(f"{what} must have rows that do not overlap")
        ld = cols
    return ld


def _rows(t, what, rows_map=None, div=1, f32=False):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must have 2 dimensions")
    return RowsStruct(t.data_ptr(), None if rows_map is None else rows_map.data_ptr(),
                      _strided(shape, t.stride(), what), shape[0], shape[1], div, _dtype(t, what, f32))


def _experts(t, what, f32=False):
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{what} must have 3 dimensions")
    E, N, K = shape
    ld = _strided(shape, stride, what)
    return ExpertsStruct(t.data_ptr(), ld, stride[0] if E > 1 else N * ld, E, N, K, _dtype(t, what, f32))


def _one(t, what, f32=False):
    """A matrix as a single expert's."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must have 2 dimensions")
    ld = _strided(shape, t.stride(), what)
    return ExpertsStruct(t.data_ptr(), ld, shape[0] * ld, 1, shape[0], shape[1], _dtype(t, what, f32))


def _ints(t, what, n=None):
    if t is None:
        return None
    if t.dtype != _torch().int32 or t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous one-dimensional int32 tensor")
    if n is not None and t.numel() != n:
        raise ValueError(f"{what} must have {n} elements")
    return t


def _count(x, x_rows, y_rows, *names):
    """The call's rows: the maps' length, or the input's rows."""
    n = [t.numel() for t in (x_rows, y_rows) if t is not None]
    if len(n) == 2 and n[0] != n[1]:
        raise ValueError(f"{names[0]} and {names[1]} must have the same length")
    return n[0] if n else x.shape[0]


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


def _run(dev, stream, call):
    """call(stream handle) with dev current and, where the caller names a
    stream, that stream current, so that what call allocates lives on it."""
    torch = _torch()
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("the stream must be on the tensors' device")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if dev == torch.cuda.current_device():
        return call(_current_stream(dev))
    with torch.cuda.device(dev):
        return call(torch.cuda.current_stream(dev).cuda_stream)


def _scratch(ws, need, dev):
    """(the tensor, its address, its bytes)"""
    torch = _torch()
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not ws.is_contiguous() or ws.dtype != torch.uint8:
        raise ValueError("ws must be a contiguous uint8 tensor")
    return ws, ws.data_ptr(), ws.numel()


def expert_matmul_workspace_bytes(op: int, E: int, R: int, N: int, K: int) -> int:
    """Workspace of an expert product (op MATMUL, MATMUL_DX or MATMUL_DW) over
    R rows, experts of N x K."""
    return int(lib().moe_expert_matmul_workspace_bytes(op, E, R, N, K))


def _expert_rows(fn, op, a, w, offsets, a_rows, a_div, c_rows, c, out_dtype, ws, stream, names):
    torch = _torch()
    an, cn = names
    dev = _device(a, w, offsets, a_rows, c_rows, c, ws)
    _ints(a_rows, f"{an}_rows")
    _ints(c_rows, f"{cn}_rows")
    R = _count(a, a_rows, c_rows, f"{an}_rows", f"{cn}_rows")
    if a_rows is None and R > a.shape[0]:
        raise ValueError(f"{cn}_rows must not be longer than {an}")
    ws_ = _experts(w, "w")
    _ints(offsets, "offsets", ws_.E + 1)
    n_out, n_in = (ws_.K, ws_.N) if op == MATMUL_DX else (ws_.N, ws_.K)
    ar = _rows(a, an, a_rows, a_div)
    if ar.cols != n_in or a.dtype != w.dtype:
        raise ValueError(f"{an} must have {n_in} columns of w's type")

    def call(s):
        nonlocal c
        if c is None:
            c = torch.empty((R, n_out), dtype=out_dtype or a.dtype, device=dev)
        elif out_dtype is not None and c.dtype != out_dtype:
            raise ValueError(f"{cn} is not of out_dtype")
        cr = _rows(c, cn, c_rows, 1, f32=True)
        scratch, p, n = _scratch(ws, expert_matmul_workspace_bytes(op, ws_.E, R, ws_.N, ws_.K), dev)
        _check(getattr(lib(), fn)(C.byref(ar), C.byref(ws_), offsets.data_ptr(), R, C.byref(cr), p, n, s), fn)
        return c
    return _run(dev, stream, call)


def expert_matmul(x, w, offsets, x_rows=None, x_div=1, y_rows=None, y=None, out_dtype=None, ws=None, stream=None):
    """y[r] = W_e x[r] for the rows r of expert e, offsets[e] <= r < offsets[e+1].

    x [n, K], w [E, N, K], offsets int32 [E + 1] (bucket's).  x_rows int32 [R]:
    row r is x[x_rows[r] // x_div] (bucket's perm with x_div = k gathers each
    pair's token); y_rows int32 [R]: row r goes to y[y_rows[r]] (perm: pair
    order).  Without them row r is row r.  An entry outside the matrix reads as
    zeros, or is not written.  Returns y [R, N] in out_dtype (default x's;
    float32 allowed); its rows that no group's row is written to are left as
    they were, undefined where this call allocates y."""
    return _expert_rows("moe_expert_matmul", MATMUL, x, w, offsets, x_rows, x_div, y_rows, y, out_dtype, ws, stream,
                        ("x", "y"))


def expert_matmul_dx(dy, w, offsets, dy_rows=None, dy_div=1, dx_rows=None, dx=None, out_dtype=None, ws=None,
                     stream=None):
    """dx[r] = W_e^T dy[r], the gradient of expert_matmul's x for each of the
    R rows (dy [n, N] -> dx [R, K]); maps as in expert_matmul."""
    return _expert_rows("moe_expert_matmul_dx", MATMUL_DX, dy, w, offsets, dy_rows, dy_div, dx_rows, dx, out_dtype, ws,
                        stream, ("dy", "dx"))


def expert_matmul_dw(dy, x, offsets, dy_rows=None, dy_div=1, x_rows=None, x_div=1, dw=None, out_dtype=None,
                     accumulate=False, ws=None, stream=None):
    """dW_e = sum over e's rows r of dy[r] x[r]^T, the gradient of
    expert_matmul's w: dw [E, N, K] (0 for an expert without rows; added to
    what dw holds if accumulate); maps as in expert_matmul."""
    torch = _torch()
    dev = _device(dy, x, offsets, dy_rows, x_rows, dw, ws)
    _ints(dy_rows, "dy_rows")
    _ints(x_rows, "x_rows")
    n = [t.shape[0] if m is None else m.numel() for t, m in ((dy, dy_rows), (x, x_rows))]
    if n[0] != n[1]:
        raise ValueError("dy and x must give the same number of rows")
    if dy.dtype != x.dtype:
        raise ValueError("dy and x must be of one type")
    E = _ints(offsets, "offsets").numel() - 1
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    dr, xr = _rows(dy, "dy", dy_rows, dy_div), _rows(x, "x", x_rows, x_div)

    def call(s):
        nonlocal dw
        if dw is None:
            dw = torch.empty((E, dr.cols, xr.cols), dtype=out_dtype or x.dtype, device=dev)
        elif out_dtype is not None and dw.dtype != out_dtype:
            raise ValueError("dw is not of out_dtype")
        d = _experts(dw, "dw", f32=True)
        if (d.E, d.N, d.K) != (E, dr.cols, xr.cols):
            raise ValueError(f"dw must be [{E}, {dr.cols}, {xr.cols}]")
        scratch, p, nb = _scratch(ws, expert_matmul_workspace_bytes(MATMUL_DW, E, n[0], d.N, d.K), dev)
        _check(lib().moe_expert_matmul_dw(C.byref(dr), C.byref(xr), offsets.data_ptr(), n[0], C.byref(d),
                                          1 if accumulate else 0, p, nb, s), "moe_expert_matmul_dw")
        return dw
    return _run(dev, stream, call)


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}")
    return ACTS[act]


def _ref(s):
    return None if s is None else C.byref(s)


def linear(x, w, bias=None, act="none", residual=None, keep_pre=False, y=None, pre=None, out_dtype=None, ws=None,
           stream=None):
    """y = act(x w^T + bias) + residual.  x [T, K], w [N, K], bias [N],
    residual [T, N] (x's type or float32); act: a key of ACTS.  Returns (y, pre): y [T, N] in out_dtype
    (default x's), pre the value before act (x's type, for linear_backward) if keep_pre or given, else
    None.  y may be the residual itself."""
    torch = _torch()
    code = _act(act)
    dev = _device(x, w, bias, residual, y, pre, ws)
    we = _one(w, "w")
    xr = _rows(x, "x")
    T, N = x.shape[0], we.N
    if xr.cols != we.K or x.dtype != w.dtype:
        raise ValueError(f"x must have {we.K} columns of w's type")
    if bias is not None and (tuple(bias.shape) != (N,) or bias.dtype != x.dtype or (N > 1 and bias.stride(0) != 1)):
        raise ValueError(f"bias must be a contiguous tensor of {N} values of x's type")
    rr = None if residual is None else _rows(residual, "residual", f32=True)

    def call(s):
        nonlocal y, pre
        if y is None:
            y = torch.empty((T, N), dtype=out_dtype or x.dtype, device=dev)
        elif out_dtype is not None and y.dtype != out_dtype:
            raise ValueError("y is not of out_dtype")
        if pre is None and keep_pre:
            pre = torch.empty((T, N), dtype=x.dtype, device=dev)
        yr, pr = _rows(y, "y", f32=True), None if pre is None else _rows(pre, "pre")
        scratch, p, n = _scratch(ws, int(lib().moe_linear_workspace_bytes(T, N, we.K)), dev)
        for m, name in ((rr, "residual"), (yr, "y"), (pr, "pre")):
            if m is not None and (m.rows, m.cols) != (T, N):
                raise ValueError(f"{name} must be [{T}, {N}]")
        _check(lib().moe_linear(C.byref(xr), C.byref(we), None if bias is None else bias.data_ptr(), code, _ref(rr),
                                _ref(pr), C.byref(yr), p, n, s), "moe_linear")
        return y, pre
    return _run(dev, stream, call)


def linear_backward(dy, x, w, act="none", pre=None, dx=None, dw=None, db=None, need_dx=True, need_dw=True,
                    need_db=False, out_dtype=None, ws=None, stream=None):
    """Gradients of linear: with dz = dy act'(pre), (dx, dw, db) = (dz w,
    dz^T x, column sums of dz), None for what is not needed (given outputs are
    needed); new ones in out_dtype (default x's).  The residual's gradient is
    dy."""
    torch = _torch()
    code = _act(act)
    if code and pre is None:
        raise ValueError("pre is needed with an activation")
    dev = _device(dy, x, w, pre, dx, dw, db, ws)
    we = _one(w, "w")
    T, N, K = dy.shape[0], we.N, we.K
    for t, shape, name in ((dy, (T, N), "dy"), (x, (T, K), "x"), (pre if code else None, (T, N), "pre"),
                           (dx, (T, K), "dx"), (dw, (N, K), "dw"), (db, (N,), "db")):
        if t is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}")
    if x.dtype != w.dtype or dy.dtype != w.dtype or (code and pre.dtype != w.dtype):
        raise ValueError("dy, x and pre must be of w's type")
    if db is not None and N > 1 and db.stride(0) != 1:
        raise ValueError("db must be contiguous")
    dyr, xr, pr = _rows(dy, "dy"), _rows(x, "x"), _rows(pre, "pre") if code else None

    def call(s):
        nonlocal dx, dw, db
        dt = out_dtype or x.dtype
        if dx is None and need_dx:
            dx = torch.empty((T, K), dtype=dt, device=dev)
        if dw is None and need_dw:
            dw = torch.empty((N, K), dtype=dt, device=dev)
        if db is None and need_db:
            db = torch.empty((N,), dtype=dt, device=dev)
        dxr = None if dx is None else _rows(dx, "dx", f32=True)
        dwe = None if dw is None else _one(dw, "dw", f32=True)
        scratch, p, n = _scratch(ws, int(lib().moe_linear_backward_workspace_bytes(T, N, K)), dev)
        _check(lib().moe_linear_backward(C.byref(dyr), C.byref(xr), C.byref(we), code, _ref(pr), _ref(dxr), _ref(dwe),
                                         None if db is None else db.data_ptr(),
                                         F32 if db is None else _dtype(db, "db", True), p, n, s),
               "moe_linear_backward")
        return dx, dw, db
    return _run(dev, stream, call)


def swiglu(gate, up, h=None, stream=None):
    """h = silu(gate) * up, all [R, I] with any row stride (gate and up may be
    the halves of one product's output).  h may be gate or up."""
    torch = _torch()
    dev = _device(gate, up, h)
    g, u = _rows(gate, "gate"), _rows(up, "up")

    def call(s):
        nonlocal h
        if h is None:
            h = torch.empty(gate.shape, dtype=gate.dtype, device=dev)
        hr = _rows(h, "h")
        _same((gate, up, h), "gate, up and h")
        _check(lib().moe_swiglu(C.byref(g), C.byref(u), C.byref(hr), s), "moe_swiglu")
        return h
    return _run(dev, stream, call)


def swiglu_backward(dh, gate, up, dgate=None, dup=None, stream=None):
    """Gradients of swiglu: (dgate, dup).  Without them given, both are views
    of one new [R, 2 I] matrix, gate's half first."""
    torch = _torch()
    dev = _device(dh, gate, up, dgate, dup)
    if (dgate is None) != (dup is None):
        raise ValueError("dgate and dup are given together")
    d, g, u = _rows(dh, "dh"), _rows(gate, "gate"), _rows(up, "up")

    def call(s):
        nonlocal dgate, dup
        if dgate is None:
            both = torch.empty((gate.shape[0], 2 * gate.shape[1]), dtype=gate.dtype, device=dev)
            dgate, dup = both[:, :gate.shape[1]], both[:, gate.shape[1]:]
        dg, du = _rows(dgate, "dgate"), _rows(dup, "dup")
        _same((dh, gate, up, dgate, dup), "dh, gate, up, dgate and dup")
        _check(lib().moe_swiglu_backward(C.byref(d), C.byref(g), C.byref(u), C.byref(dg), C.byref(du), s),
               "moe_swiglu_backward")
        return dgate, dup
    return _run(dev, stream, call)


def _same(ts, names):
    shape, dtype = ts[0].shape, ts[0].dtype
    for t in ts:
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{names} must be of one shape and type")


def _weights(w, k, n, what):
    """(T, k) of a combine over n expert rows."""
    torch = _torch()
    if w is not None:
        if w.dim() != 2 or w.dtype != torch.float32 or not w.is_contiguous():
            raise ValueError("w must be a contiguous float32 [T, k]")
        if k is not None and k != w.shape[1]:
            raise ValueError("k is not w's")
        k = w.shape[1]
        if w.shape[0] * k != n:
            raise ValueError(f"{what} must have T * k rows")
        return w.shape[0], k
    if k is None or k < 1 or n % k:
        raise ValueError(f"without w, k is needed and {what} has T * k rows")
    return n // k, k


def combine(o, w=None, k=None, residual=None, y=None, out_dtype=None, stream=None):
    """y[t] = sum_j w[t, j] o[t k + j] + residual[t].  o [T k, H], w float32
    [T, k] (None: ones, with k given), residual [T, H] (o's type or float32).
    y [T, H] in out_dtype (default the residual's, else o's; o's or float32); y
    may be the residual itself."""
    torch = _torch()
    dev = _device(o, w, residual, y)
    T, k = _weights(w, k, o.shape[0], "o")
    orow = _rows(o, "o")
    rr = None if residual is None else _rows(residual, "residual", f32=True)

    def call(s):
        nonlocal y
        if y is None:
            y = torch.empty((T, o.shape[1]), device=dev,
                            dtype=out_dtype or (o.dtype if residual is None else residual.dtype))
        elif out_dtype is not None and y.dtype != out_dtype:
            raise ValueError("y is not of out_dtype")
        yr = _rows(y, "y", f32=True)
        for m, name in ((rr, "residual"), (yr, "y")):
            if m is not None and (m.rows, m.cols) != (T, o.shape[1]):
                raise ValueError(f"{name} must be [{T}, {o.shape[1]}]")
        _check(lib().moe_combine(C.byref(orow), None if w is None else w.data_ptr(), T, k, _ref(rr), C.byref(yr), s),
               "moe_combine")
        return y
    return _run(dev, stream, call)


def combine_backward(dy, o=None, w=None, k=None, d_o=None, dw=None, need_do=True, need_dw=True, stream=None):
    """Gradients of combine: (d_o, dw) with d_o[t k + j] = w[t, j] dy[t] (o's
    type) and dw[t, j] = <dy[t], o[t k + j]> (float32); None for one not
    needed.  Without o (then need_dw = False) d_o is of dy's type.  The
    residual's gradient is dy.  d_o may be o itself."""
    torch = _torch()
    need_dw = need_dw or dw is not None
    need_do = need_do or d_o is not None
    if need_dw and o is None:
        raise ValueError("dw needs o")
    dev = _device(dy, o, w, d_o, dw)
    if o is None and w is None and k is None:
        raise ValueError("without o and w, k is needed")
    n = o.shape[0] if o is not None else dy.shape[0] * (w.shape[1] if w is not None else k)
    T, k = _weights(w, k, n, "o")
    yr = _rows(dy, "dy", f32=True)
    orow = None if o is None else _rows(o, "o")

    def call(s):
        nonlocal d_o, dw
        if d_o is None and need_do:
            d_o = torch.empty((T * k, dy.shape[1]), dtype=dy.dtype if o is None else o.dtype, device=dev)
        if dw is None and need_dw:
            dw = torch.empty((T, k), dtype=torch.float32, device=dev)
        dr = None if d_o is None else _rows(d_o, "d_o")
        for m, rows, name in ((yr, T, "dy"), (orow, T * k, "o"), (dr, T * k, "d_o")):
            if m is not None and (m.rows, m.cols) != (rows, dy.shape[1]):
                raise ValueError(f"{name} must be [{rows}, {dy.shape[1]}]")
        if dw is not None and (tuple(dw.shape) != (T, k) or dw.dtype != torch.float32 or not dw.is_contiguous()):
            raise ValueError(f"dw must be a contiguous float32 [{T}, {k}]")
        if dr is None and dw is None:
            return None, None
        _check(lib().moe_combine_backward(C.byref(yr), _ref(orow), None if w is None else w.data_ptr(), T, k, _ref(dr),
                                          None if dw is None else dw.data_ptr(), s), "moe_combine_backward")
        return d_o, dw
    return _run(dev, stream, call)
