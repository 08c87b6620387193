"""The norms around a block on the GPU against float64.  Bounds: _rows8.py, per
element, from the float32 sums' and products' roundings."""
import pytest

import _rows8 as r8
from _gpu import require_gpu, say, torch
from test_gpu_experts import BF, F32, HF, check, gen, place, rnd

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def vec(g, n, dtype):
    v = torch.randn(n, generator=g).to(dtype)
    return v.cuda(), v.double()


def case(T, H, dtype, stream, gate, pad=0, shift=0, seed=0):
    """Device tensors and their float64 values."""
    g = gen(T + H + seed)
    d = {"o": rnd(g, T, H, dtype=dtype, scale=0.5, pad=pad, shift=shift), "residual": rnd(g, T, H, dtype=stream, scale=2.0, pad=pad, shift=shift),
         "wa": vec(g, H, dtype), "wb": vec(g, H, dtype),
         "gate": None if gate == "none" else vec(g, H, dtype) if gate == "channel" else rnd(g, T, H, dtype=dtype, pad=pad),
         "ds": rnd(g, T, H, dtype=stream, pad=pad), "dn": rnd(g, T, H, dtype=dtype, pad=pad, shift=shift)}
    dev = {k: None if v is None else v[0] for k, v in d.items()}
    val = {k: torch.ones(1, dtype=r8.F64) if v is None else v[1] for k, v in d.items()}
    return dev, val


SHAPES = [(1, 1, 0, 0), (3, 7, 1, 1), (1, 7168, 0, 0), (5, 64, 0, 0), (70, 513, 3, 1), (9, 2047, 0, 0), (600, 520, 8, 8),
          (530, 2048, 0, 0), (2, 8200, 0, 0), (3, 16384, 0, 0), (515, 7168, 0, 0), (33, 4104, 0, 0), (1500, 100, 0, 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("dtype,stream", [(BF, BF), (HF, HF), (BF, F32), (HF, F32)], ids=["bf16", "fp16", "bf16-fp32", "fp16-fp32"])
def test_forward(bm, shape, gate, dtype, stream):
    T, H, pad, shift = shape
    d, v = case(T, H, dtype, stream, gate, pad, shift)
    say(f"[norm] forward {shape} {gate} {dtype} {stream}")
    kw = dict(w_after=d["wa"], gate=d["gate"], scale=0.875, w_before=d["wb"], eps=EPS)
    s, n = bm.block_norm(d["o"], d["residual"], **kw)
    ws, wn, es, en = r8.norm_bounds(v["o"], v["residual"], v["wa"], v["gate"], 0.875, v["wb"], EPS, stream, dtype)
    check(s, ws, es, "s")
    check(n, wn, en, "n")
    assert s.dtype == stream and n.dtype == dtype
    # one without the other; into given ones; over the residual and o themselves
    s1, none = bm.block_norm(d["o"], d["residual"], need_n=False, **kw)
    assert none is None and torch.equal(s1, s)
    none, n1 = bm.block_norm(d["o"], d["residual"], need_s=False, **kw)
    assert none is None and torch.equal(n1, n)
    s2 = place(torch.full((T, H), 7.0, dtype=stream), pad, shift, hold=3.0)
    n2 = place(torch.full((T, H), 7.0, dtype=dtype), pad, shift, hold=3.0)
    bm.block_norm(d["o"], d["residual"], s=s2, n=n2, **kw)
    assert torch.equal(s2, s) and torch.equal(n2, n)
    if pad and T > 1:
        assert (n2.as_strided((T - 1, pad), (H + pad, 1), shift + H) == 3).all()
    o, res = d["o"].clone(), d["residual"].clone()
    assert bm.block_norm(o, res, s=res, n=o, **kw)[0] is res
    assert torch.equal(res, s) and torch.equal(o, n)
    # the norm before the first block alone; the norm after without a stream
    if gate == "none":
        one = torch.ones(1, dtype=r8.F64)
        none, n3 = bm.block_norm(None, d["residual"], w_before=d["wb"], eps=EPS, need_s=False)
        _, wn, _, en = r8.norm_bounds(None, v["residual"], one, one, 1.0, v["wb"], EPS, stream, dtype)
        check(n3, wn, en, "norm before")
        s4, none = bm.block_norm(d["o"], eps=EPS, need_n=False)
        ws, _, es, _ = r8.norm_bounds(v["o"], None, one, one, 1.0, one, EPS, dtype, dtype)
        check(s4, ws, es, "norm after, no weights, no stream")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("dtype,stream,dw", [(BF, BF, BF), (HF, HF, F32), (BF, F32, F32)], ids=["bf16", "fp16", "bf16-fp32"])
def test_backward(bm, shape, gate, dtype, stream, dw):
    T, H, pad, shift = shape
    d, v = case(T, H, dtype, stream, gate, pad, shift, 1)
    say(f"[norm] backward {shape} {gate} {dtype} {stream}")
    kw = dict(w_after=d["wa"], gate=d["gate"], scale=0.875, w_before=d["wb"], eps=EPS, out_dtype=dw)
    got = bm.block_norm_backward(d["dn"], d["ds"], d["residual"], d["o"], **kw)
    want, bound = r8.norm_backward_bounds(v["dn"], v["ds"], v["residual"], v["o"], v["wa"], v["gate"], 0.875, v["wb"], EPS,
                                          dtype, stream, dw)
    for name in ("d_o", "dresidual", "dw_after", "dw_before"):
        check(getattr(got, name), want[name], bound[name], name)
    assert got.d_o.dtype == dtype and got.dresidual.dtype == stream and got.dw_after.dtype == dw
    if gate == "none":
        assert got.dgate is None
    else:
        name = "dgate" if gate == "token" else "dgate_sum"
        check(got.dgate, want[name], bound[name], name)
        assert got.dgate.dtype == (dtype if gate == "token" else dw)
    # one at a time, and over their inputs
    lone = bm.block_norm_backward(d["dn"], d["ds"], d["residual"], d["o"], need_dw=False, need_dresidual=False, **kw)
    assert torch.equal(lone.d_o, got.d_o) and lone.dresidual is None and lone.dw_after is None and lone.dgate is None
    ds, o = d["ds"].clone(), d["o"].clone()
    over = bm.block_norm_backward(d["dn"], ds, d["residual"], o, dresidual=ds, d_o=o, **kw)
    assert over.d_o is o and torch.equal(o, got.d_o) and torch.equal(ds, got.dresidual) and torch.equal(over.dw_before, got.dw_before)
    if gate == "token":
        gt = d["gate"].clone()
        bm.block_norm_backward(d["dn"], d["ds"], d["residual"], d["o"], dgate=gt, **{**kw, "gate": gt})
        assert torch.equal(gt, got.dgate)
    again = bm.block_norm_backward(d["dn"], d["ds"], d["residual"], d["o"], **kw)
    assert all(x is None or torch.equal(x, y) for x, y in zip(again, got))


@pytest.mark.parametrize("T,H", [(1, 7168), (5, 100), (530, 2050)])
def test_backward_parts(bm, T, H):
    """The first block's norm (no o), the last block's (no dn), a stream with no
    later use (no ds)."""
    d, v = case(T, H, BF, F32, "channel", seed=2)
    one = torch.ones(1, dtype=r8.F64)
    say(f"[norm] backward's parts {T} {H}")

    def compare(got, names, *args):
        want, bound = r8.norm_backward_bounds(*args, EPS, BF, F32 if args[1] is not None else BF, BF)
        for name in names:
            check(getattr(got, name.replace("_sum", "")), want[name], bound[name], name)
    got = bm.block_norm_backward(d["dn"], d["ds"], d["residual"], w_before=d["wb"], eps=EPS)
    assert got.d_o is None and got.dw_after is None and got.dgate is None
    compare(got, ("dresidual", "dw_before"), v["dn"], v["ds"], v["residual"], None, one, one, 1.0, v["wb"])
    got = bm.block_norm_backward(None, d["ds"], None, d["o"], w_after=d["wa"], gate=d["gate"], eps=EPS)
    assert got.dw_before is None
    compare(got, ("d_o", "dresidual", "dw_after", "dgate_sum"), None, v["ds"], None, v["o"], v["wa"], v["gate"], 1.0, one)
    got = bm.block_norm_backward(d["dn"], None, d["residual"], d["o"], eps=EPS, scale=2.0)
    compare(got, ("d_o", "dresidual"), v["dn"], None, v["residual"], v["o"], one, one, 2.0, one)
    assert got.dresidual.dtype == BF and got.dw_before is None
    # the gradient at ones of weights that the forward call had not
    w = torch.empty(H, dtype=F32, device="cuda")
    got = bm.block_norm_backward(d["dn"], None, d["residual"], d["o"], eps=EPS, dw_before=w, scale=2.0, need_do=False, need_dresidual=False)
    want, bound = r8.norm_backward_bounds(v["dn"], None, v["residual"], v["o"], one, one, 2.0, one, EPS, BF, BF, F32)
    check(w, want["dw_before"], bound["dw_before"], "dw_before at ones")


@pytest.mark.parametrize("big", [1e25, 3e38])
def test_squares_that_leave_float32(bm, big):
    """Rows whose squares' sum is infinite in float32 and small ones beside them."""
    T, H = 4, 300
    g = gen(11)
    o = torch.randn(T, H, generator=g).to(BF)
    o[1] = (torch.rand(H, generator=g) * 2 - 1).to(BF) * big
    o[2] = torch.randn(H, generator=g).to(BF) * 1e-25
    o[3] = 0
    w = torch.randn(H, generator=g).to(BF)
    say(f"[norm] squares past float32 {big}")
    one = torch.ones(1, dtype=r8.F64)
    s, none = bm.block_norm(o.cuda(), w_after=w.cuda(), eps=EPS, need_n=False, stream_dtype=F32)
    ws, _, es, _ = r8.norm_bounds(o.double(), None, w.double(), one, 1.0, one, EPS, F32, BF)
    check(s, ws, es + 1e-40, "s")
    assert (s[3] == 0).all()
    none, n = bm.block_norm(None, o.cuda(), w_before=w.cuda(), eps=EPS, need_s=False)
    _, wn, _, en = r8.norm_bounds(None, o.double(), one, one, 1.0, w.double(), EPS, BF, BF)
    check(n, wn, en + 1e-40, "n")
    dn = torch.randn(T, H, generator=g).to(BF)
    got = bm.block_norm_backward(dn.cuda(), None, o.cuda(), o.cuda(), w_after=w.cuda(), w_before=w.cuda(), eps=EPS, out_dtype=F32)
    # (1 / rms of the large row is near float32's smallest normal value, where what is taken times it keeps less)
    want, bound = r8.norm_backward_bounds(dn.double(), None, o.double(), o.double(), w.double(), one, 1.0, w.double(), EPS, BF, BF, F32)
    for name in ("d_o", "dresidual", "dw_after", "dw_before"):
        check(getattr(got, name), want[name], bound[name] + 1e-36, name)


def test_values_that_are_not_finite(bm):
    """An infinity or NaN makes its own row NaN where the formula does, and the
    token sums; no other row."""
    T, H = 6, 130
    o = torch.randn(T, H, generator=gen(1)).to(BF)
    o[1, 5], o[4, 129] = float("inf"), float("nan")
    r = torch.randn(T, H, generator=gen(2)).to(BF)
    s, n = (t.cpu() for t in bm.block_norm(o.cuda(), r.cuda(), eps=EPS))
    bad = torch.tensor([False, True, False, False, True, False])
    assert torch.isnan(n[bad]).all() and torch.isnan(s[4]).all() and torch.isnan(s[1, 5])
    assert torch.isfinite(s[~bad]).all() and torch.isfinite(n[~bad]).all()
    got = bm.block_norm_backward(r.cuda(), r.cuda(), r.cuda(), o.cuda(), eps=EPS)
    assert torch.isfinite(got.d_o[~bad.cuda()]).all() and torch.isfinite(got.dresidual).all()


def test_no_tokens(bm):
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    s, n = bm.block_norm(e, e, w_after=w, w_before=w, gate=w)
    assert s.shape == n.shape == (0, 64)
    got = bm.block_norm_backward(e, e, e, e, w_after=w, w_before=w, gate=w, out_dtype=F32)
    assert got.d_o.shape == (0, 64) and all((t == 0).all() for t in (got.dw_after, got.dw_before, got.dgate))
