"""Binding of the expert layer's operators in 8 bits and of the norms around a
block (bitmoe.h, "The 16-bit expert layer's rows in 8 bits" and "The norms around
a block"): argument checks, output and workspace allocation, and the call, with
the conventions of the 16-bit layer's binding (experts.py).
"""
from __future__ import annotations

import struct
from typing import Any, NamedTuple

from ._lib import I8, _check, _torch, lib
from .experts import (_current_stream, _device, _dtype_code, _elsewhere, _ints, _one_type, _output, _rows, _scratch,
                      _strided, _vector)

BLOCKS = (0, 32, 64, 128)

# bitmoe_rows8 and bitmoe_experts8 as bytes
_ROWS8 = struct.Struct("@PPqiiiiPqii")
_EXPERTS8 = struct.Struct("@PqqiiiiPq")


class Rows8(NamedTuple):
    """Rows in 8 bits.  codes int8 [R, C] (experts' weights: [E, N, K]), unit
    stride along the last dimension; scale float32: block 0 (one scale a row)
    [R] ([E, N]), else [R, blocks of a row], unit stride along the last
    dimension.  A code stands for code * scale."""
    codes: Any
    scale: Any
    block: int = 0


class BlockNormGrads(NamedTuple):
    """Gradients of block_norm; None for one that was not needed."""
    d_o: Any
    dresidual: Any
    dw_after: Any
    dgate: Any
    dw_before: Any


def _rows8(q, what, shape, rows_map=None, div=1):
    """A bitmoe_rows8; shape: what the call needs (None for any number of
    rows)."""
    codes, scale, block = q
    torch = _torch()
    if codes.dim() != 2 or codes.dtype != torch.int8:
        raise ValueError(f"{what}'s codes must be int8 with 2 dimensions")
    if block not in BLOCKS:
        raise ValueError(f"{what}'s block must be one of {BLOCKS}")
    n, cols = codes.shape
    if cols != shape[1] or (shape[0] is not None and n != shape[0]):
        raise ValueError(f"{what} must be [{'n' if shape[0] is None else shape[0]}, {shape[1]}]")
    ld = _strided(n, cols, codes.stride(), f"{what}'s codes")
    if scale.dtype != torch.float32:
        raise TypeError(f"{what}'s scale must be float32")
    want = (n, -(-cols // block)) if block else (n,)
    if tuple(scale.shape) != want:
        raise ValueError(f"{what}'s scale must be {list(want)}")
    if block:
        ls = _strided(n, want[1], scale.stride(), f"{what}'s scale")
    else:
        ls = scale.stride(0) if n > 1 else 1
        if ls < 1:
            raise ValueError(f"{what}'s scale must have values that do not overlap")
    try:
        return _ROWS8.pack(codes.data_ptr(), 0 if rows_map is None else rows_map.data_ptr(), ld, n, cols, div, I8,
                           scale.data_ptr(), ls, block, 0)
    except struct.error:
        raise ValueError(f"{what} or its map's divisor is too large") from None


def _experts8(q, what):
    """(bitmoe_experts8, E, N, K): codes [E, N, K], or [N, K] as a single
    expert's."""
    codes, scale, block = q
    torch = _torch()
    if codes.dtype != torch.int8 or codes.dim() not in (2, 3):
        raise ValueError(f"{what}'s codes must be int8 with 2 or 3 dimensions")
    if block != 0 or scale.dtype != torch.float32 or tuple(scale.shape) != tuple(codes.shape[:-1]):
        raise ValueError(f"{what}'s scale must be float32, one for each row")
    E, N, K = codes.shape if codes.dim() == 3 else (1, *codes.shape)
    ld = _strided(N, K, codes.stride(), f"{what}'s codes")
    if N > 1 and scale.stride(-1) != 1:
        raise ValueError(f"{what}'s scale must have unit stride along its last dimension")
    return _EXPERTS8.pack(codes.data_ptr(), ld, codes.stride(0) if E > 1 else N * ld, E, N, K, I8,
                          scale.data_ptr(), scale.stride(0) if E > 1 else N), E, N, K


def _new_rows8(rows, cols, block, dev):
    """(a new Rows8, its bitmoe_rows8: nothing of it needs a check)"""
    if block not in BLOCKS:
        raise ValueError(f"block must be one of {BLOCKS}")
    torch = _torch()
    codes = torch.empty((rows, cols), dtype=torch.int8, device=dev)
    n = -(-cols // block) if block else 1
    scale = torch.empty((rows, n) if block else (rows,), dtype=torch.float32, device=dev)
    return Rows8(codes, scale, block), _ROWS8.pack(codes.data_ptr(), 0, cols, rows, cols, 1, I8, scale.data_ptr(), n, block, 0)


def _given_rows8(out, shape, block):
    if out.block != block:
        raise ValueError("out is not of block")
    return _rows8(out, "out", shape)


def quantize_rows(x, block=0, out=None, stream=None):
    """Rows8 of x [R, C] (bfloat16, float16 or float32) with a scale for `block`
    columns, 32, 64 or 128, or (0) for the row; into `out` if given.  x [E, N, K]
    (contiguous experts) gives experts' weights with a scale for each of their
    rows, codes [E, N, K] and scale [E, N]."""
    given = () if out is None else (out.codes, out.scale)
    dev = _device(x, *given)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return quantize_rows(x, block, out)
    if x.dim() == 3:
        E, N, K = x.shape
        if block or out is not None or (E > 1 and N and x.stride(0) != N * x.stride(1)):
            raise ValueError("experts' weights must be contiguous, take block 0 and no out")
        q = quantize_rows(x.reshape(E * N, K) if not x.numel() else x.view(E * N, K))
        return Rows8(q.codes.view(E, N, K), q.scale.view(E, N), 0)
    xr = _rows(x, "x", f32=True)
    if out is None:
        out, qr = _new_rows8(*x.shape, block, dev)
    else:
        qr = _given_rows8(out, x.shape, block)
    _check(lib().moe_quantize_rows(xr, qr, _current_stream(dev)), "moe_quantize_rows")
    return out


def dequantize_rows(q, dtype=None, y=None, stream=None):
    """The values of a Rows8: y [R, C] = code * scale in `dtype` (bfloat16,
    float16 or float32; default y's, else bfloat16)."""
    dev = _device(q.codes, q.scale, y)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return dequantize_rows(q, dtype, y)
    shape = tuple(q.codes.shape)
    qr = _rows8(q, "q", (None, shape[-1]))
    y = _output(y, shape, dtype or _torch().bfloat16, dev, "y", dtype)
    _check(lib().moe_dequantize_rows(qr, _rows(y, "y", shape, f32=True), _current_stream(dev)), "moe_dequantize_rows")
    return y


def expert_matmul_i8_workspace_bytes(E: int, R: int, N: int, K: int) -> int:
    """Workspace of an expert product in 8 bits."""
    return int(lib().moe_expert_matmul_i8_workspace_bytes(E, R, N, K))


def expert_matmul_i8(x, w, offsets=None, x_rows=None, x_div=1, y_rows=None, y=None, out_dtype=None, ws=None,
                     stream=None):
    """expert_matmul with both operands in 8 bits: y[r] = W_e x[r], the codes'
    products summed exactly, times x[r]'s scale, times each output's.

    x: Rows8 [n, K], one scale a row (quantize_rows); w: Rows8 [E, N, K] with a
    scale for each row of each expert, or [N, K] (without offsets: one product
    of all rows).  Maps, offsets and y as in expert_matmul; y [R, N] in
    out_dtype (bfloat16, float16 or float32; default y's, else bfloat16)."""
    dev = _device(x.codes, x.scale, w.codes, w.scale, offsets, x_rows, y_rows, y, ws)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return expert_matmul_i8(x, w, offsets, x_rows, x_div, y_rows, y, out_dtype, ws)
    we, E, N, K = _experts8(w, "w")
    if x.block != 0:
        raise ValueError("x must have one scale a row")
    R = _ints(x_rows, "x_rows") if x_rows is not None else None
    if y_rows is not None:
        n = _ints(y_rows, "y_rows")
        if R is None:
            R = n
            if n > x.codes.shape[0]:
                raise ValueError("y_rows must not be longer than x")
        elif n != R:
            raise ValueError("x_rows and y_rows must have the same length")
    elif R is None:
        R = x.codes.shape[0]
    if offsets is not None:
        _ints(offsets, "offsets", E + 1)
    elif E != 1:
        raise ValueError("experts need offsets")
    xr = _rows8(x, "x", (None, K), x_rows, x_div)
    ungrouped = y is None and y_rows is not None and offsets is not None
    y = _output(y, (R, N), out_dtype or _torch().bfloat16, dev, "y", out_dtype)
    yr = _rows(y, "y", (None, N), y_rows, 1, f32=True)
    L = lib()
    hold, p, n = _scratch(ws, L.moe_expert_matmul_i8_workspace_bytes(E, R, N, K), dev)
    s = _current_stream(dev)
    off = None if offsets is None else offsets.data_ptr()
    if ungrouped:
        _check(L.moe_expert_clear_ungrouped(off, E, R, yr, s), "moe_expert_clear_ungrouped")
    _check(L.moe_expert_matmul_i8(xr, we, off, R, yr, p, n, s), "moe_expert_matmul_i8")
    return y


def swiglu_rows8(gate, up, block=0, out=None, stream=None):
    """h = silu(gate) * up straight into 8 bits (Rows8 [R, I], as
    quantize_rows'): with block 0 for a down projection by expert_matmul_i8, with
    another block to be kept and read back by dequantize_rows."""
    given = () if out is None else (out.codes, out.scale)
    dev = _device(gate, up, *given)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return swiglu_rows8(gate, up, block, out)
    g = _rows(gate, "gate")
    _one_type("gate and up", gate, up)
    if out is None:
        out, qr = _new_rows8(*gate.shape, block, dev)
    else:
        qr = _given_rows8(out, gate.shape, block)
    _check(lib().moe_swiglu_rows8(g, _rows(up, "up", gate.shape), qr, _current_stream(dev)), "moe_swiglu_rows8")
    return out


def swiglu_checkpoint(gate, up, block=64, h=None, gate8=None, up8=None, stream=None):
    """swiglu, and its inputs in 8 bits for swiglu_checkpoint_backward: (h, gate8,
    up8), the last two Rows8 of `block` 32, 64 or 128 (halves of one new tensor
    of codes and one of scales, if not given)."""
    given = [t for q in (gate8, up8) if q is not None for t in (q.codes, q.scale)]
    dev = _device(gate, up, h, *given)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return swiglu_checkpoint(gate, up, block, h, gate8, up8)
    if (gate8 is None) != (up8 is None):
        raise ValueError("gate8 and up8 are given together")
    g = _rows(gate, "gate")
    shape = R, I = gate.shape
    _one_type("gate, up and h", gate, up, *(() if h is None else (h,)))
    if gate8 is None:
        if block not in BLOCKS[1:]:
            raise ValueError(f"block must be one of {BLOCKS[1:]}")
        torch = _torch()
        n = -(-I // block)
        codes = torch.empty((2, R, I), dtype=torch.int8, device=dev)
        scale = torch.empty((2, R, n), dtype=torch.float32, device=dev)
        (gc, uc), (gs, us) = codes.unbind(0), scale.unbind(0)
        gate8, up8 = Rows8(gc, gs, block), Rows8(uc, us, block)
        at, sat = codes.data_ptr(), scale.data_ptr()
        gr = _ROWS8.pack(at, 0, I, R, I, 1, I8, sat, n, block, 0)
        ur = _ROWS8.pack(at + R * I, 0, I, R, I, 1, I8, sat + 4 * R * n, n, block, 0)
    else:
        gr, ur = _rows8(gate8, "gate8", shape), _rows8(up8, "up8", shape)
    h = _output(h, shape, gate.dtype, dev, "h")
    _check(lib().moe_swiglu_checkpoint(g, _rows(up, "up", shape), _rows(h, "h", shape), gr, ur, _current_stream(dev)),
           "moe_swiglu_checkpoint")
    return h, gate8, up8


def swiglu_checkpoint_backward(dh, gate8, up8, dgate=None, dup=None, need_h=False, h=None, stream=None):
    """Gradients of swiglu at what swiglu_checkpoint kept: (dgate, dup, h), h (if
    needed or given, else None) being swiglu of what was kept, for the down
    projection's weights' gradient.  All of dh's type; dgate and dup are views of
    one new [R, 2 I] matrix if not given."""
    dev = _device(dh, gate8.codes, gate8.scale, up8.codes, up8.scale, dgate, dup, h)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return swiglu_checkpoint_backward(dh, gate8, up8, dgate, dup, need_h, h)
    if (dgate is None) != (dup is None):
        raise ValueError("dgate and dup are given together")
    d = _rows(dh, "dh")
    shape = dh.shape
    if dgate is None:
        both = _torch().empty((shape[0], 2 * shape[1]), dtype=dh.dtype, device=dev)
        dgate, dup = both.split(shape[1], 1) if shape[1] else (both, both)
    if h is None and need_h:
        h = _torch().empty(shape, dtype=dh.dtype, device=dev)
    _one_type("dh, dgate, dup and h", dh, dgate, dup, *(() if h is None else (h,)))
    _check(lib().moe_swiglu_checkpoint_backward(d, _rows8(gate8, "gate8", shape), _rows8(up8, "up8", shape),
                                                _rows(dgate, "dgate", shape), _rows(dup, "dup", shape),
                                                None if h is None else _rows(h, "h", shape), _current_stream(dev)),
           "moe_swiglu_checkpoint_backward")
    return dgate, dup, h


def _gate(gate, T, H, what, f32=False):
    """A gate's bitmoe_rows: [H], or [T, H]."""
    if gate is None:
        return None
    if gate.dim() == 1:
        if gate.shape[0] != H or (H > 1 and gate.stride(0) != 1):
            raise ValueError(f"{what} must be contiguous, [{H}] or [{T}, {H}]")
        gate = gate.view(1, H)
        return _rows(gate, what, (1, H), f32=f32)
    return _rows(gate, what, (T, H))


def block_norm(o, residual=None, w_after=None, gate=None, scale=1.0, w_before=None, eps=1e-6, s=None, n=None,
               need_s=True, need_n=True, stream_dtype=None, stream=None):
    """The norm after a block, its gate, the residual stream and the norm before
    the next block: (s, n) with

        s = scale * residual + gate * (o / rms(o) * w_after)
        n = s / rms(s) * w_before,    rms(v) = sqrt(mean(v^2) + eps)

    o [T, H], weights [H], gate [H] or [T, H], of one 16-bit type; residual and s
    [T, H] of that type or float32 (s: stream_dtype, default the residual's, else
    o's).  What is None is left out: o (the norm before the first block), residual
    (0), weights and gate (1).  Of s and n, one that is not needed is None; s may
    be the residual itself, n may be o."""
    need_s, need_n = need_s or s is not None, need_n or n is not None
    if (o is None and residual is None) or not (need_s or need_n):
        raise ValueError("block_norm needs o or residual, and s or n")
    dev = _device(*(t for t in (o, residual) if t is not None), w_after, gate, w_before, s, n)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return block_norm(o, residual, w_after, gate, scale, w_before, eps, s, n, need_s, need_n, stream_dtype)
    torch = _torch()
    first = residual if o is None else o
    shape = T, H = first.shape if first.dim() == 2 else (0, 0)
    dtype = next((t.dtype for t in (o, n, w_before) if t is not None), first.dtype)
    if dtype == torch.float32:
        raise ValueError("o, weights or n must say which 16-bit type n has")
    if o is None and not need_n:
        raise ValueError("block_norm needs o or n")
    typed = [t for t in (o, gate, w_after, w_before, n) if t is not None]
    if typed:
        _one_type("o, gate, weights and n", *typed)
    orow = None if o is None else _rows(o, "o")
    rr = None if residual is None else _rows(residual, "residual", shape, f32=True)
    if need_s:
        s = _output(s, shape, stream_dtype or first.dtype if residual is None else stream_dtype or residual.dtype, dev,
                    "s", stream_dtype)
    if need_n:
        n = _output(n, shape, dtype, dev, "n")
    _check(lib().moe_block_norm(orow, None if w_after is None else _vector(w_after, H, "w_after"),
                                _gate(gate, T, H, "gate"), rr, scale,
                                None if s is None else _rows(s, "s", shape, f32=True),
                                None if w_before is None else _vector(w_before, H, "w_before"), eps,
                                None if n is None else _rows(n, "n", shape), _current_stream(dev)), "moe_block_norm")
    return s, n


def block_norm_backward_workspace_bytes(T: int, H: int) -> int:
    """Workspace of block_norm_backward."""
    return int(lib().moe_block_norm_backward_workspace_bytes(T, H))


def block_norm_backward(dn=None, ds=None, s=None, o=None, w_after=None, gate=None, scale=1.0, w_before=None, eps=1e-6,
                        d_o=None, dresidual=None, dw_after=None, dgate=None, dw_before=None, need_do=True,
                        need_dresidual=True, need_dw=True, out_dtype=None, ws=None, stream=None):
    """Gradients of block_norm, a BlockNormGrads: dn [T, H] is n's gradient, ds
    [T, H] that of s from the stream's later uses (one may be None), s and o what
    the forward call gave and had (s with dn; o None if it had none), the rest as
    there.  dresidual is of ds's type (without it dn's: for the last norm of a
    stream in float32, give one in float32) if not given; dw_after,
    dw_before [H] and the gradient of a gate [H] are sums over tokens in out_dtype
    (default the 16-bit type, or that of a given one; float32 allowed), that of a
    gate [T, H] is of its type.  need_dw: the weights' and the gate's, where the
    call has them.  dresidual may be ds itself, d_o may be o or dn, dgate [T, H] the
    gate."""
    if dn is None and ds is None:
        raise ValueError("block_norm_backward needs dn or ds")
    dev = _device(*(t for t in (dn, ds) if t is not None), s, o, w_after, gate, w_before, d_o, dresidual, dw_after, dgate,
                  dw_before, ws)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return block_norm_backward(dn, ds, s, o, w_after, gate, scale, w_before, eps, d_o, dresidual, dw_after,
                                       dgate, dw_before, need_do, need_dresidual, need_dw, out_dtype, ws)
    torch = _torch()
    first = ds if dn is None else dn
    if dn is None and o is None:
        raise ValueError("block_norm_backward needs dn or o")
    shape = T, H = first.shape if first.dim() == 2 else (0, 0)
    dtype = (o if dn is None else dn).dtype
    _one_type("dn, o, gate, weights and d_o", *(t for t in (dn, o, gate, w_after, w_before, d_o) if t is not None))
    dnr = None if dn is None else _rows(dn, "dn")
    dsr = None if ds is None else _rows(ds, "ds", f32=True)
    if o is not None and (need_do or d_o is not None):
        d_o = _output(d_o, shape, dtype, dev, "d_o")
    if need_dresidual or dresidual is not None:
        dresidual = _output(dresidual, shape, first.dtype if ds is None else ds.dtype, dev, "dresidual")
    given = next((t.dtype for t in (dw_after, dw_before) if t is not None), None)
    out_dtype = out_dtype or given or dtype
    if w_after is not None and need_dw or dw_after is not None:
        dw_after = _output(dw_after, (H,), out_dtype, dev, "dw_after", out_dtype)
    if w_before is not None and need_dw or dw_before is not None:
        dw_before = _output(dw_before, (H,), out_dtype, dev, "dw_before", out_dtype)
    if gate is not None and need_dw or dgate is not None:
        if gate is None:
            raise ValueError("dgate needs gate")
        dgate = _output(dgate, tuple(gate.shape), out_dtype if gate.dim() == 1 else dtype, dev, "dgate")
        if dgate.dim() != gate.dim():
            raise ValueError("dgate must have the gate's shape")
    L = lib()
    hold, p, n = _scratch(ws, L.moe_block_norm_backward_workspace_bytes(T, H), dev)
    opt = lambda t, what, f32: None if t is None else _rows(t, what, shape, f32=f32)  # noqa: E731
    vec = lambda t, what: None if t is None else _vector(t, H, what)  # noqa: E731
    _check(L.moe_block_norm_backward(dnr, dsr, opt(s, "s", True), opt(o, "o", False), vec(w_after, "w_after"),
                                     _gate(gate, T, H, "gate"), scale, vec(w_before, "w_before"), eps,
                                     opt(d_o, "d_o", False), opt(dresidual, "dresidual", True),
                                     vec(dw_after, "dw_after"), _gate(dgate, T, H, "dgate", f32=True),
                                     vec(dw_before, "dw_before"), _dtype_code(out_dtype, "out_dtype", True), p, n,
                                     _current_stream(dev)), "moe_block_norm_backward")
    return BlockNormGrads(d_o, dresidual, dw_after, dgate, dw_before)
