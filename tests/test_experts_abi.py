"""Refusals of the 16-bit expert layer's calls, without a GPU: every check
runs on the host before a launch, and a call that passes them all with no rows
queues nothing."""
import ctypes as C

import pytest
import torch

import bit_moe_amd as bm
from bit_moe_amd import _lib
from bit_moe_amd._lib import BF16, EINVAL, EUNSUPPORTED, EWORKSPACE, F16, F32, ExpertsStruct, RowsStruct

P = 4096            # an aligned address that nothing dereferences


def rows(n=8, cols=16, data=P, map=None, ld=None, div=1, dtype=BF16):
    return C.byref(RowsStruct(data, map, cols if ld is None else ld, n, cols, div, dtype))


def experts(E=4, N=32, K=16, data=P, ld=None, stride=None, dtype=BF16):
    ld = K if ld is None else ld
    return C.byref(ExpertsStruct(data, ld, N * ld if stride is None else stride, E, N, K, dtype))


BAD_ROWS = [dict(data=None), dict(data=P + 1), dict(ld=4), dict(cols=24), dict(n=-1), dict(n=7), dict(dtype=7),
            dict(map=P, div=0), dict(map=P + 2), dict(dtype=F16)]
BAD_EXPERTS = [(dict(data=None), EINVAL), (dict(data=P + 1), EINVAL), (dict(ld=8), EINVAL), (dict(stride=100), EINVAL),
               (dict(E=0), EINVAL), (dict(N=0), EINVAL), (dict(E=1025), EUNSUPPORTED),
               (dict(N=(1 << 18) + 1), EUNSUPPORTED), (dict(dtype=5), EINVAL)]


@pytest.mark.parametrize("dx", [False, True])
def test_expert_matmul_refusals(dx):
    L = bm.lib()
    f = L.moe_expert_matmul_dx if dx else L.moe_expert_matmul
    ci, co = (32, 16) if dx else (16, 32)

    def call(a={}, w={}, off=P, R=8, y={}):
        return f(rows(**{"cols": ci, **a}), experts(**w), off, R, rows(**{"cols": co, **y}), None, 0, None)
    assert call(R=0) == 0
    assert call(a=dict(data=None), y=dict(data=None), off=None, R=0) == 0
    for bad in BAD_ROWS:
        assert call(a=bad) == EINVAL, bad
        assert call(y=bad) == EINVAL, bad
    assert call(a=dict(dtype=F32)) == EINVAL
    for bad, code in BAD_EXPERTS:
        assert call(w=bad) == code, bad
    assert call(w=dict(dtype=F32)) == EINVAL
    assert call(off=None) == EINVAL and call(off=P + 2) == EINVAL
    assert call(R=-1) == EINVAL and call(R=(1 << 24) + 1) == EUNSUPPORTED
    assert f(None, experts(), P, 8, rows(cols=co), None, 0, None) == EINVAL
    assert f(rows(cols=ci), None, P, 8, rows(cols=co), None, 0, None) == EINVAL
    assert f(rows(cols=ci), experts(), P, 8, None, None, 0, None) == EINVAL


def test_expert_matmul_dw_refusals():
    f = bm.lib().moe_expert_matmul_dw

    def call(dy={}, x={}, off=P, R=8, dw={}):
        return f(rows(**{"cols": 32, **dy}), rows(**x), off, R, experts(**dw), 0, None, 0, None)
    for bad in BAD_ROWS:
        assert call(dy=bad) == EINVAL and call(x=bad) == EINVAL, bad
    for bad, code in BAD_EXPERTS:
        assert call(dw=bad) == code, bad
    assert call(dy=dict(dtype=F32), x=dict(dtype=F32)) == EINVAL
    assert call(off=None) == EINVAL and call(R=(1 << 24) + 1) == EUNSUPPORTED


def test_workspace_sizes_and_checks():
    L = bm.lib()
    for op in (bm.MATMUL, bm.MATMUL_DX, bm.MATMUL_DW):
        for E, R, N, K in ((1, 1, 1, 1), (256, 8, 2048, 7168), (32, 32768, 7168, 2048), (1024, 1 << 24, 64, 64)):
            assert bm.expert_matmul_workspace_bytes(op, E, R, N, K) % 256 == 0
        assert bm.expert_matmul_workspace_bytes(op, 0, 8, 16, 16) == 0
    assert bm.expert_matmul_workspace_bytes(3, 4, 8, 16, 16) == 0
    need = L.moe_linear_backward_workspace_bytes(8, 32, 16)
    assert need > 0 and need % 256 == 0

    def back(ws=P, n=need, db=None):
        return L.moe_linear_backward(rows(cols=32), rows(), experts(E=1), 4, rows(cols=32), rows(), experts(E=1), db,
                                     F32, ws, n, None)
    assert back(ws=None) == EWORKSPACE and back(n=need - 1) == EWORKSPACE and back(ws=P + 16) == EWORKSPACE
    assert back(db=P + 2) == EINVAL


def test_linear_refusals():
    L = bm.lib()

    def call(x={}, w={}, bias=P, act=2, res={}, pre={}, y={}):
        return L.moe_linear(rows(**x), experts(**{"E": 1, **w}), bias, act,
                            None if res is None else rows(**{"cols": 32, **res}),
                            None if pre is None else rows(**{"cols": 32, **pre}), rows(**{"cols": 32, **y}), None, 0, None)
    empty = dict(n=0, data=None)
    assert call(x=empty, res=empty, pre=empty, y=empty) == 0
    assert call(x=empty, res=None, pre=None, y=empty, bias=None) == 0
    for bad in BAD_ROWS + [dict(map=P)]:
        if bad != dict(n=7):
            assert call(x=bad) == EINVAL, bad
        assert call(res=bad) == EINVAL and call(pre=bad) == EINVAL and call(y=bad) == EINVAL, bad
    assert call(pre=dict(dtype=F32)) == EINVAL
    assert call(act=5) == EINVAL and call(act=-1) == EINVAL and call(bias=P + 1) == EINVAL
    assert call(w=dict(E=2)) == EINVAL

    def back(dy={}, x={}, w={}, act=2, pre={}, dx={}, dw={}):
        return L.moe_linear_backward(rows(**{"cols": 32, **dy}), rows(**x), experts(**{"E": 1, **w}), act,
                                     None if pre is None else rows(**{"cols": 32, **pre}), rows(**dx),
                                     experts(**{"E": 1, **dw}), None, F32, None, 0, None)
    for bad in BAD_ROWS + [dict(map=P)]:
        if bad != dict(n=7):
            assert back(dy=bad) == EINVAL, bad
        assert back(x=bad) == EINVAL and back(pre=bad) == EINVAL and back(dx=bad) == EINVAL, bad
    assert back(pre=None) == EINVAL and back(act=9) == EINVAL
    assert back(dw=dict(K=17)) == EINVAL and back(dw=dict(E=2)) == EINVAL and back(w=dict(E=3)) == EINVAL
    # nothing asked for: nothing queued
    assert L.moe_linear_backward(rows(cols=32), None, experts(E=1), 0, None, None, None, None, F32, None, 0, None) == 0


def test_rows_call_refusals():
    L = bm.lib()
    r = rows
    assert L.moe_swiglu(r(n=0), r(n=0), r(n=0), None) == 0
    assert L.moe_swiglu(None, r(), r(), None) == EINVAL
    for bad in BAD_ROWS + [dict(map=P), dict(dtype=F32)]:
        assert L.moe_swiglu(r(), r(**bad), r(), None) == EINVAL, bad
        assert L.moe_swiglu(r(), r(), r(**bad), None) == EINVAL, bad
        for i in (0, 2, 3, 4):
            a = [r()] * 5
            a[i] = r(**bad)
            assert L.moe_swiglu_backward(*a, None) == EINVAL, bad
    # combine: 4 tokens of 2 experts
    y = lambda **kw: r(**{"n": 4, **kw})  # noqa: E731
    assert L.moe_combine(r(n=0), None, 0, 2, None, y(n=0), None) == 0
    assert L.moe_combine(r(), P, 4, 17, None, y(), None) == EUNSUPPORTED
    assert L.moe_combine(r(), P, 4, 0, None, y(), None) == EINVAL
    assert L.moe_combine(r(), P, 5, 2, None, r(n=5), None) == EINVAL
    assert L.moe_combine(r(), P + 2, 4, 2, None, y(), None) == EINVAL
    assert L.moe_combine(None, P, 4, 2, None, y(), None) == EINVAL
    assert L.moe_combine(r(dtype=F32), P, 4, 2, None, y(), None) == EINVAL
    assert L.moe_combine(r(), P, 1 << 24, 2, None, y(), None) == EUNSUPPORTED
    for bad in (dict(data=None), dict(ld=4), dict(cols=24), dict(dtype=F16), dict(map=P), dict(n=3)):
        assert L.moe_combine(r(), P, 4, 2, y(**bad), y(), None) == EINVAL, bad
        assert L.moe_combine(r(), P, 4, 2, None, y(**bad), None) == EINVAL, bad
        assert L.moe_combine_backward(y(**bad), r(), P, 4, 2, r(), P, None) == EINVAL, bad
    assert L.moe_combine_backward(y(), r(), P, 4, 2, None, None, None) == EINVAL
    assert L.moe_combine_backward(y(), None, P, 4, 2, r(), P, None) == EINVAL
    assert L.moe_combine_backward(y(), r(), P, 4, 2, r(dtype=F16), None, None) == EINVAL
    assert L.moe_combine_backward(y(), r(), P, 4, 2, r(), P + 1, None) == EINVAL


def test_binding_refuses_what_is_not_on_the_gpu():
    x, w, off = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 4, 8, dtype=torch.bfloat16), torch.zeros(3)
    for f in (lambda: bm.expert_matmul(x, w, off), lambda: bm.expert_matmul_dw(x, x, off), lambda: bm.linear(x, w[0]),
              lambda: bm.linear_backward(x[:, :4], x, w[0]), lambda: bm.swiglu(x, x), lambda: bm.combine(x, k=2),
              lambda: bm.combine_backward(x, x, k=1)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        bm.linear(x, w[0], act="swish")
