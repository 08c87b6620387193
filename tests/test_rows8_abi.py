"""Refusals of the calls in 8 bits and of the block norms, without a GPU: every
check runs on the host before a launch, and a call that passes them all with no
rows queues nothing."""
import ctypes as C

import pytest
import torch

import bit_moe_amd as bm
from bit_moe_amd import experts
from bit_moe_amd import rows8 as binding
from bit_moe_amd._lib import (BF16, EINVAL, EUNSUPPORTED, EWORKSPACE, F16, F32, I8, Experts8Struct, ExpertsStruct,
                              Rows8Struct, RowsStruct)

P = 4096            # an aligned address that nothing dereferences


def rows(n=8, cols=16, data=P, map=None, ld=None, div=1, dtype=BF16):
    return C.byref(RowsStruct(data, map, cols if ld is None else ld, n, cols, div, dtype))


def rows8(n=8, cols=16, data=P, map=None, ld=None, div=1, dtype=I8, scale=P, ld_scale=None, block=0, reserved=0):
    q = RowsStruct(data, map, cols if ld is None else ld, n, cols, div, dtype)
    return C.byref(Rows8Struct(q, scale, (-(-cols // block) if block > 0 else 1) if ld_scale is None else ld_scale, block, reserved))


def experts8(E=4, N=32, K=16, data=P, ld=None, stride=None, dtype=I8, scale=P, scale_stride=None):
    ld = K if ld is None else ld
    q = ExpertsStruct(data, ld, N * ld if stride is None else stride, E, N, K, dtype)
    return C.byref(Experts8Struct(q, scale, N if scale_stride is None else scale_stride))


BAD_ROWS = [dict(data=None), dict(data=P + 1), dict(ld=4), dict(cols=24), dict(n=-1), dict(n=7), dict(dtype=7), dict(dtype=I8),
            dict(map=P)]
BAD_ROWS8 = [dict(data=None), dict(ld=4), dict(cols=24), dict(n=-1), dict(n=7), dict(dtype=BF16), dict(scale=None),
             dict(scale=P + 2), dict(ld_scale=0), dict(block=16), dict(block=-1), dict(block=256), dict(reserved=1)]


def test_structures_are_the_headers():
    assert C.sizeof(Rows8Struct) == binding._ROWS8.size == 64
    assert C.sizeof(Experts8Struct) == binding._EXPERTS8.size == 56


def test_quantize_and_dequantize_refusals():
    L = bm.lib()
    for f, ab in ((lambda x={}, q={}: L.moe_quantize_rows(rows(**x), rows8(**q), None), True),
                  (lambda x={}, q={}: L.moe_dequantize_rows(rows8(**q), rows(**x), None), False)):
        for bad in BAD_ROWS:
            if ab and bad in (dict(n=7), dict(cols=24)):        # the call's own sizes: the codes do not agree
                continue
            assert f(x=bad) == EINVAL, bad
        for bad in BAD_ROWS8 + [dict(map=P)]:
            if not ab and bad == dict(n=7):
                continue
            assert f(q=bad) == EINVAL, bad
        assert f(x=dict(n=0, data=None), q=dict(n=0, data=None, scale=None)) == 0
        assert f(x=dict(n=(1 << 24) + 1), q=dict(n=(1 << 24) + 1)) == EUNSUPPORTED
        wide = dict(cols=(1 << 18) + 1)
        assert f(x=wide, q=wide) == EUNSUPPORTED
        assert f(x=dict(cols=0), q=dict(cols=0)) == EINVAL
        # every block's scales have their place
        for block, cols, need in ((32, 33, 2), (64, 128, 2), (128, 300, 3)):
            assert f(x=dict(n=0, cols=cols), q=dict(n=0, cols=cols, block=block, ld_scale=need)) == 0
            assert f(x=dict(n=0, cols=cols), q=dict(n=0, cols=cols, block=block, ld_scale=need - 1)) == EINVAL
    assert L.moe_quantize_rows(None, rows8(), None) == EINVAL and L.moe_quantize_rows(rows(), None, None) == EINVAL
    assert L.moe_dequantize_rows(None, rows(), None) == EINVAL and L.moe_dequantize_rows(rows8(), None, None) == EINVAL


def test_swiglu_rows8_refusals():
    f = lambda g={}, u={}, q={}: bm.lib().moe_swiglu_rows8(rows(**g), rows(**u), rows8(**q), None)  # noqa: E731
    assert f(dict(n=0), dict(n=0), dict(n=0)) == 0
    for bad in BAD_ROWS + [dict(dtype=F16), dict(dtype=F32)]:
        assert f(u=bad) == EINVAL, bad
    for bad in BAD_ROWS8:
        assert f(q=bad) == EINVAL, bad
    assert f(g=dict(dtype=F32), u=dict(dtype=F32)) == EINVAL
    assert bm.lib().moe_swiglu_rows8(None, rows(), rows8(), None) == EINVAL


def test_checkpoint_refusals():
    L = bm.lib()
    b = dict(block=64)

    def forward(g={}, u={}, h={}, a={}, c={}):
        return L.moe_swiglu_checkpoint(rows(**g), rows(**u), rows(**h), rows8(**{**b, **a}), rows8(**{**b, **c}), None)

    def backward(d={}, a={}, c={}, dg={}, du={}, h={}):
        return L.moe_swiglu_checkpoint_backward(rows(**d), rows8(**{**b, **a}), rows8(**{**b, **c}), rows(**dg), rows(**du),
                                                None if h is None else rows(**h), None)
    no = dict(n=0)
    assert forward(no, no, no, no, no) == 0 and backward(no, no, no, no, no, no) == 0 == backward(no, no, no, no, no, None)
    for bad in BAD_ROWS + [dict(dtype=F16), dict(dtype=F32)]:
        assert forward(u=bad) == forward(h=bad) == EINVAL, bad
        assert backward(dg=bad) == backward(du=bad) == backward(h=bad) == EINVAL, bad
    for bad in BAD_ROWS8 + [dict(block=0), dict(block=32, ld_scale=1)]:
        assert forward(a=bad) == forward(c=bad) == EINVAL, bad
        assert backward(a=bad) == backward(c=bad) == EINVAL, bad
    assert forward(g=dict(dtype=F32), u=dict(dtype=F32), h=dict(dtype=F32)) == EINVAL
    assert L.moe_swiglu_checkpoint(None, rows(), rows(), rows8(**b), rows8(**b), None) == EINVAL
    assert L.moe_swiglu_checkpoint_backward(None, rows8(**b), rows8(**b), rows(), rows(), None, None) == EINVAL


def test_expert_matmul_i8_refusals():
    L = bm.lib()

    def call(x={}, w={}, off=P, R=8, y={}, ws=None, n=0):
        return L.moe_expert_matmul_i8(rows8(**x), experts8(**w), off, R, rows(**{"cols": 32, **y}), ws, n, None)
    assert call(R=0) == 0 and call(x=dict(data=None, scale=None), y=dict(data=None), R=0) == 0
    for bad in BAD_ROWS8 + [dict(map=P, div=0), dict(map=P + 2), dict(block=32)]:
        assert call(x=bad) == EINVAL, bad
    for bad in [d for d in BAD_ROWS if d != dict(map=P)] + [dict(map=P, div=0), dict(map=P + 2)]:
        assert call(y=bad) == EINVAL, bad
    for bad, code in [(dict(data=None), EINVAL), (dict(ld=8), EINVAL), (dict(stride=100), EINVAL), (dict(E=0), EINVAL),
                      (dict(N=0), EINVAL), (dict(E=1025), EUNSUPPORTED), (dict(dtype=BF16), EINVAL), (dict(scale=None), EINVAL),
                      (dict(scale=P + 1), EINVAL), (dict(scale_stride=31), EINVAL)]:
        assert call(w=bad) == code, bad
    k = 1 << 17
    assert call(x=dict(cols=k), w=dict(K=k)) == EUNSUPPORTED
    assert call(x=dict(cols=k - 1), w=dict(K=k - 1), R=0) == 0
    assert call(off=None) == EINVAL and call(off=P + 2) == EINVAL and call(off=None, w=dict(E=1), R=0) == 0
    assert call(R=-1) == EINVAL and call(R=(1 << 24) + 1) == EUNSUPPORTED
    for args in ((None, experts8(), P, 8, rows(cols=32)), (rows8(), None, P, 8, rows(cols=32)), (rows8(), experts8(), P, 8, None)):
        assert L.moe_expert_matmul_i8(*args, None, 0, None) == EINVAL


def test_block_norm_refusals():
    L = bm.lib()
    none = object()
    opt = lambda d: None if d is none else rows(**d)  # noqa: E731

    def call(o={}, wa=P, gate={}, res={}, s={}, wb=P, eps=1e-6, n={}):
        return L.moe_block_norm(opt(o), wa, opt(gate), opt(res), 1.0, opt(s), wb, eps, opt(n), None)
    no = dict(n=0)
    assert call(o=no, gate=no, res=no, s=no, n=no) == 0
    assert call(o=no, gate=dict(n=1), res=no, s=no, n=no) == 0
    assert call(o=none, wa=None, gate=none, res=no, s=none, n=no) == 0
    assert call(o=no, wa=None, gate=none, res=none, s=no, wb=None, n=none) == 0
    for bad in BAD_ROWS:
        if bad in (dict(n=7), dict(cols=24), dict(n=-1)):
            assert call(res=bad) == call(s=bad) == call(n=bad) == EINVAL, bad
            assert call(gate=bad) == EINVAL, bad
            continue
        for name in ("o", "gate", "res", "s", "n"):
            assert call(**{name: bad}) == EINVAL, (name, bad)
    for name in ("gate", "n", "res", "s"):
        assert call(**{name: dict(dtype=F16)}) == EINVAL
    assert call(o=dict(dtype=F32)) == call(gate=dict(dtype=F32)) == call(n=dict(dtype=F32)) == EINVAL
    assert call(res=dict(dtype=F32), s=dict(dtype=F32), n=none, wa=P + 1) == EINVAL
    assert call(wb=P + 1) == EINVAL and call(s=none, n=none) == EINVAL and call(o=none, wa=None, gate=none, res=none) == EINVAL
    assert call(o=none, gate=none) == EINVAL and call(o=none, wa=None) == EINVAL       # a weight, a gate without o
    assert call(o=none, wa=None, gate=none, n=none) == EINVAL
    for eps in (0.0, -1e-6, 1e-31, float("nan"), float("inf")):
        assert call(eps=eps) == EINVAL, eps
    big = dict(cols=16385)
    assert call(o=big, gate=big, res=big, s=big, n=big) == EUNSUPPORTED


def test_block_norm_backward_refusals():
    L = bm.lib()
    none = object()
    opt = lambda d: None if d is none else rows(**d)  # noqa: E731
    need = L.moe_block_norm_backward_workspace_bytes(8, 16)
    assert need > 0 and need % 256 == 0 and L.moe_block_norm_backward_workspace_bytes(8, 16385) == 0
    assert L.moe_block_norm_backward_workspace_bytes(-1, 16) == 0

    def call(dn={}, ds={}, s={}, o={}, wa=P, gate={}, wb=P, eps=1e-6, d_o={}, dr={}, dwa=P, dg={}, dwb=P, dt=BF16, ws=P, n=need):
        return L.moe_block_norm_backward(opt(dn), opt(ds), opt(s), opt(o), wa, opt(gate), 1.0, wb, eps, opt(d_o), opt(dr), dwa,
                                         opt(dg), dwb, dt, ws, n, None)
    out = dict(d_o=none, dr=none, dwa=None, dg=none, dwb=None)
    assert call(**out) == 0                                                            # nothing is wanted
    assert call(ws=None) == call(n=need - 1) == call(ws=P + 128) == EWORKSPACE
    for bad in BAD_ROWS:
        if bad in (dict(n=7), dict(cols=24), dict(n=-1)):
            for name in ("ds", "s", "o", "gate", "d_o", "dr", "dg"):
                assert call(**{name: bad}) == EINVAL, (name, bad)
            continue
        for name in ("dn", "ds", "s", "o", "gate", "d_o", "dr", "dg"):
            assert call(**{name: bad}) == EINVAL, (name, bad)
    for name in ("ds", "s", "o", "gate", "d_o", "dr", "dg"):
        assert call(**{name: dict(dtype=F16)}) == EINVAL
    for name in ("dn", "o", "gate", "d_o", "dg"):
        assert call(**{name: dict(dtype=F32)}) == EINVAL
    assert call(dt=F16) == call(dt=7) == call(dt=I8) == EINVAL and call(dwa=P + 2, dt=F32) == call(dwb=P + 1) == EINVAL
    assert call(wa=P + 1) == call(wb=P + 1) == EINVAL
    assert call(s=none) == EINVAL and call(dn=none) == EINVAL and call(dn=none, ds=none) == EINVAL
    assert call(o=none) == EINVAL and call(gate=none) == EINVAL
    assert call(dn=none, wb=None, dwb=None, o=none, wa=None, gate=none, d_o=none, dwa=None, dg=none) == EINVAL
    assert call(gate=dict(n=1), dg=dict(n=1, dtype=F16)) == EINVAL
    assert call(dg=dict(n=1)) == EINVAL
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == EINVAL


class OnGpu(torch.Tensor):
    """A tensor on the CPU that says it is on a device."""
    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class Allocates:
    """torch, whose new tensors are such."""
    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *args, device=None, **kw):
        return torch.empty(*args, **kw).as_subclass(OnGpu)


def test_binding_refusals(monkeypatch):
    """What the binding refuses before it calls the library."""
    monkeypatch.setattr(binding, "_elsewhere", lambda dev, stream: None)
    monkeypatch.setattr(binding, "_current_stream", lambda dev: None)
    for module in (binding, experts):
        monkeypatch.setattr(module, "_torch", lambda: Allocates())
    x = on_gpu(8, 64)
    q = bm.Rows8(on_gpu(8, 64, dtype=torch.int8), on_gpu(8, dtype=torch.float32))
    w = bm.Rows8(on_gpu(4, 16, 64, dtype=torch.int8), on_gpu(4, 16, dtype=torch.float32))
    off = on_gpu(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        bm.quantize_rows(torch.zeros(8, 64))
    for bad in (lambda: bm.quantize_rows(x, block=16), lambda: bm.quantize_rows(x, out=bm.Rows8(*q[:2], 32)),
                lambda: bm.quantize_rows(x, out=bm.Rows8(q.codes[:, :8], q.scale)),
                lambda: bm.quantize_rows(x, out=bm.Rows8(q.codes, q.scale[:7])),
                lambda: bm.quantize_rows(x[0]), lambda: bm.quantize_rows(x.t()), lambda: bm.quantize_rows(on_gpu(2, 8, 64), block=32),
                lambda: bm.quantize_rows(x, block=32, out=bm.Rows8(q.codes, on_gpu(8, 3, dtype=torch.float32), 32)),
                lambda: bm.dequantize_rows(bm.Rows8(x, q.scale)), lambda: bm.dequantize_rows(q, y=on_gpu(8, 63)),
                lambda: bm.dequantize_rows(q, dtype=torch.float16, y=x),
                lambda: bm.expert_matmul_i8(q, w), lambda: bm.expert_matmul_i8(q, w, off[:4]),
                lambda: bm.expert_matmul_i8(bm.Rows8(q.codes, on_gpu(8, 2, dtype=torch.float32), 32), w, off),
                lambda: bm.expert_matmul_i8(q, bm.Rows8(w.codes, w.scale[:, :8]), off),
                lambda: bm.expert_matmul_i8(q, bm.Rows8(w.codes[:, :, :32], w.scale), off),
                lambda: bm.expert_matmul_i8(q, w, off, x_rows=on_gpu(8, dtype=torch.int32), y_rows=on_gpu(7, dtype=torch.int32)),
                lambda: bm.expert_matmul_i8(q, w, off, y_rows=on_gpu(9, dtype=torch.int32)),
                lambda: bm.expert_matmul_i8(q, w, off, y=on_gpu(8, 16), out_dtype=torch.float32),
                lambda: bm.swiglu_rows8(x, on_gpu(8, 64, dtype=torch.float16)), lambda: bm.swiglu_rows8(x, x, block=48),
                lambda: bm.swiglu_checkpoint(x, x, block=0), lambda: bm.swiglu_checkpoint(x, x, gate8=bm.Rows8(*q[:2], 64)),
                lambda: bm.swiglu_checkpoint_backward(x, q, q, dgate=x),
                lambda: bm.block_norm(None), lambda: bm.block_norm(x, need_s=False, need_n=False),
                lambda: bm.block_norm(x, gate=on_gpu(63)), lambda: bm.block_norm(x, gate=on_gpu(7, 64)),
                lambda: bm.block_norm(x, w_after=on_gpu(63)), lambda: bm.block_norm(x, w_after=on_gpu(64, dtype=torch.float16)),
                lambda: bm.block_norm(None, on_gpu(8, 64, dtype=torch.float32)), lambda: bm.block_norm(None, x, need_n=False),
                lambda: bm.block_norm(x, s=x, stream_dtype=torch.float32), lambda: bm.block_norm_backward(None, None),
                lambda: bm.block_norm_backward(x, x, x, x, dgate=x), lambda: bm.block_norm_backward(None, x),
                lambda: bm.block_norm_backward(x, x, x, x, gate=on_gpu(64), dgate=on_gpu(1, 64)),
                lambda: bm.block_norm_backward(x, x, x, x, w_after=on_gpu(64), dw_after=on_gpu(64), out_dtype=torch.float32)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        bm.quantize_rows(on_gpu(8, 64, dtype=torch.float64))
    with pytest.raises(TypeError):
        bm.quantize_rows(x, out=bm.Rows8(q.codes, on_gpu(8)))
