"""What the 16-bit expert layer's calls accept, without a GPU: a call that
passes every check asks for its workspace (BITMOE_EWORKSPACE) or, with no rows,
queues nothing."""
import ctypes as C
import os
import re

import pytest

import bit_moe_amd as bm
from bit_moe_amd import experts as ex
from bit_moe_amd._lib import BF16, EINVAL, EUNSUPPORTED, EWORKSPACE, F16, F32, ExpertsStruct, RowsStruct

P = 4096            # an aligned address that nothing dereferences
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bitmoe.h")


def rows(n=8, cols=16, data=P, map=None, ld=None, div=1, dtype=BF16):
    return C.byref(RowsStruct(data, map, cols if ld is None else ld, n, cols, div, dtype))


def experts(E=4, N=32, K=16, data=P, ld=None, stride=None, dtype=BF16):
    ld = K if ld is None else ld
    return C.byref(ExpertsStruct(data, ld, N * ld if stride is None else stride, E, N, K, dtype))


def test_the_bindings_acts_are_the_headers():
    src = open(HEADER).read()
    names = {m[0].lower(): int(m[1]) for m in re.findall(r"#define BITMOE_ACT_(\w+)\s+(\d+)", src)}
    assert names.pop("round_dz") == ex.ROUND_DZ
    assert names == ex.ACTS


@pytest.mark.parametrize("act", range(5))
def test_backward_with_and_without_rounded_dz(act):
    L = bm.lib()

    def back(act, ws=None, n=0, dtype=BF16):
        r = lambda cols: rows(cols=cols, dtype=dtype)  # noqa: E731
        return L.moe_linear_backward(r(32), r(16), experts(E=1, dtype=dtype), act, r(32), r(16), experts(E=1, dtype=dtype),
                                     P, F32, ws, n, None)
    need = L.moe_linear_backward_workspace_bytes(8, 32, 16)
    assert need >= 8 * 32 * 2 * 2                        # dz in two parts
    for dtype in (BF16, F16):
        assert back(act, dtype=dtype) == back(act | ex.ROUND_DZ, dtype=dtype) == EWORKSPACE
        assert back(act | ex.ROUND_DZ, P, need - 1, dtype) == EWORKSPACE
    assert back(act | 512) == EINVAL and back(5 | ex.ROUND_DZ) == EINVAL
    # the forward pass knows no such flag
    assert L.moe_linear(rows(n=0), experts(E=1), None, act | ex.ROUND_DZ, None, None, rows(n=0, cols=32), None, 0, None) == EINVAL


def test_experts_apart_by_what_the_header_says():
    """The least distance between experts that is accepted is the header's:
    up to the last element, not to the end of a padded last row."""
    assert re.search(r"ld >= K; stride >= \(N - 1\) \* ld \+ K when E > 1", open(HEADER).read())
    L = bm.lib()
    for n, k, ld in ((32, 16, 16), (32, 16, 24), (1, 16, 100)):
        for less, rc in ((0, EWORKSPACE), (1, EINVAL)):
            w = experts(N=n, K=k, ld=ld, stride=(n - 1) * ld + k - less)
            assert L.moe_expert_matmul_dw(rows(cols=n), rows(cols=k), P, 8, w, 0, None, 0, None) == rc


def test_maps_over_a_matrix_without_rows():
    """Every entry lies outside it: rows of zeros, nothing written.  No address
    is asked for (torch gives none to a tensor without elements)."""
    L = bm.lib()
    none, w = dict(n=0, data=None, map=P), experts()
    assert L.moe_expert_matmul_dw(rows(cols=32, **none), rows(), P, 8, w, 0, None, 0, None) == EWORKSPACE
    assert L.moe_expert_matmul_dw(rows(cols=32), rows(**none), P, 8, w, 0, None, 0, None) == EWORKSPACE
    for bad in (dict(n=0, data=None), dict(n=8, data=None, map=P), dict(n=8, data=P + 1, map=P)):
        assert L.moe_expert_matmul_dw(rows(cols=32, **bad), rows(), P, 8, w, 0, None, 0, None) == EINVAL, bad


def test_clear_ungrouped_refusals():
    L = bm.lib()

    def call(off=P, E=4, R=8, **kw):
        return L.moe_expert_clear_ungrouped(off, E, R, rows(**kw), None)
    assert call(R=0, off=None, n=0, data=None) == 0
    assert L.moe_expert_clear_ungrouped(P, 4, 8, None, None) == EINVAL
    for bad in (dict(off=None), dict(off=P + 2), dict(E=0), dict(R=-1), dict(n=7), dict(ld=8), dict(dtype=7), dict(data=None),
                dict(dtype=F32, data=P + 2), dict(map=P + 1), dict(map=P, div=0), dict(cols=0)):
        assert call(**bad) == EINVAL, bad
    assert call(E=1025) == EUNSUPPORTED and call(R=(1 << 24) + 1, n=1 << 25) == EUNSUPPORTED
