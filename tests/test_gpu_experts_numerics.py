"""The 16-bit expert layer's numerics where a rounding could hide in the sums:
operands of few non-zeros, so that a bound per element stays tight over any
contraction, with float32 outputs."""
import math

import pytest

import _experts as ex
import _experts_cases as cases
from _gpu import require_gpu, say, torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["gelu", "gelu_tanh", "silu"]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def sparse(n, cols, g, dtype, most=4):
    """[n, cols] with at most `most` non-zeros (powers of two) in a column."""
    m = torch.zeros(n, cols)
    for _ in range(most):
        m[torch.randint(n, (cols,), generator=g), torch.arange(cols)] = \
            2.0 ** torch.randint(-3, 2, (cols,), generator=g) * (1 - 2.0 * torch.randint(2, (cols,), generator=g))
    return m.to(dtype)


def padded(v, pad, shift):
    """v on the device, its rows `pad` elements further apart and `shift`
    elements behind an aligned address."""
    ld = v.shape[1] + pad
    buf = torch.full((shift + v.shape[0] * ld + 8,), float("nan"), dtype=v.dtype, device="cuda")
    t = buf.as_strided(v.shape, (ld, 1), shift)
    t.copy_(v)
    return t


def over(got, want, bound):
    assert torch.isfinite(got).all()
    return ((got.double() - want).abs() / (bound + 1e-300)).max().item()


# What dz = dy act'(pre) may be off by before the products: the slope's own
# evaluation, and what the two 16-bit parts of dz leave (each rounding is off by
# at most half a step, of the value and then of what that left; in float16 the
# low part's smallest step, 2^-24, stands for 2^-34 of dz, and half of it is lost)
def dz_error(dz, dy, dtype):
    ez = 2.0 ** -17 * dy.abs()
    return ez + ex.half_ulp(dtype) ** 2 * (dz.abs() + ez) + 2.0 ** -35 * (dtype == HF)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("case", cases.BACKWARD, ids=str)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_products_of_linear_backward_take_dz_whole(bm, act, case, dtype):
    T, N, K, pad, shift = case[2:]
    g = torch.Generator().manual_seed(T + N + K)
    x, w = sparse(T, K, g, dtype), sparse(N, K, g, dtype)
    pre, dy = (torch.randn(T, N, generator=g) * 2).to(dtype), torch.randn(T, N, generator=g).to(dtype)
    say(f"[experts] dz whole {act} {case} {dtype}")
    args = [padded(t, pad, shift) for t in (dy, x, w)]
    dx, dw, _ = bm.linear_backward(*args, act=act, pre=padded(pre, pad, 0), out_dtype=F32)
    dy, x, w = dy.cuda().double(), x.cuda().double(), w.cuda().double()         # (the oracle's products on the GPU)
    dz = dy * ex.act_slope(pre.cuda().double(), act)
    e = dz_error(dz, dy, dtype)
    m = dz.abs() + e
    # 4 products of each part, which together are at most 1.01 dz
    for name, got, want, err, mag in (("dx", dx, dz @ w, e @ w.abs(), m @ w.abs()),
                                      ("dw", dw, dz.t() @ x, e.t() @ x.abs(), m.t() @ x.abs())):
        worst = over(got, want, err + 1.01 * ex.sum_bound(8) * mag + 2.0 ** -24 * want.abs())
        say(f"[experts] {name}: largest error {worst:.2f} of its bound")
        assert worst <= 1, (name, worst)


@pytest.mark.parametrize("act,at", [("gelu", 1.5), ("gelu_tanh", 1.5), ("silu", 2.5)])
@pytest.mark.parametrize("shape", [(40, 64, 72), (33, 17, 35), (2048, 2048, 2048)], ids=str)
def test_linear_backward_over_the_whole_range_of_float16(bm, act, at, shape):
    """dz beyond float16's largest value, and below its smallest."""
    T, N, K = shape
    g = torch.Generator().manual_seed(N)
    pre = torch.full((T, N), at, dtype=HF)
    dy = (65504.0 * (1 - 2.0 * torch.randint(2, (T, N), generator=g))).to(HF)
    pre[T // 2:] = -0.3
    dy[T // 2:] = 2.0 ** -24 * torch.randint(-3, 4, (T - T // 2, N), generator=g).to(HF)
    x, w = sparse(T, K, g, HF, 1), sparse(N, K, g, HF, 1)
    dx, dw, db = bm.linear_backward(dy.cuda(), x.cuda(), w.cuda(), act=act, pre=pre.cuda(), out_dtype=F32, need_db=True)
    dy, x, w = dy.cuda().double(), x.cuda().double(), w.cuda().double()
    dz = dy * ex.act_slope(pre.cuda().double(), act)
    assert dz[0].abs().min() > 65520 and 0 < dz[-1].abs().max() < 2.0 ** -23
    e = dz_error(dz, dy, HF)
    for name, got, want, err in (("dx", dx, dz @ w, e @ w.abs()), ("dw", dw, dz.t() @ x, e.t() @ x.abs())):
        worst = over(got, want, err + 1.01 * ex.sum_bound(2) * want.abs())
        say(f"[experts] {name} {act} {shape}: largest error {worst:.2f} of its bound")
        assert worst <= 1, (name, worst)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_linear_backward_with_infinities(bm, dtype):
    """An infinity or NaN in dy makes what its row and column of dz reach so,
    as the formula has it, and nothing else."""
    g = torch.Generator().manual_seed(1)
    dy, x = torch.randn(64, 64, generator=g), torch.randn(64, 64, generator=g).abs() + 0.1
    w, pre = torch.randn(64, 64, generator=g).abs() + 0.1, torch.full((64, 64), 1.0)
    clean = [t.to(dtype).cuda() for t in (dy, x, w, pre)]
    dx0, dw0, _ = bm.linear_backward(*clean[:3], act="silu", pre=clean[3])
    for value in (math.inf, -math.inf, math.nan):
        bad = clean[0].clone()
        bad[5, 9] = value
        dx, dw, _ = bm.linear_backward(bad, *clean[1:3], act="silu", pre=clean[3])
        for got, was, at in ((dx, dx0, 5), (dw, dw0, 9)):
            assert (got[at].isnan() if math.isnan(value) else got[at] == value).all()
            rest = [i for i in range(64) if i != at]
            assert torch.equal(got[rest], was[rest])


@pytest.mark.parametrize("act", ["none", "relu"] + ACTS)
@pytest.mark.parametrize("shape", [(1, 64, 72), (33, 17, 35), (300, 520, 264), (2048, 1000, 2048)], ids=str)
def test_linear_backward_of_rounded_dz(bm, act, shape):
    """round_dz: the products of dz rounded to the operands' type; the same as
    without it where dz is dy or 0 anyway."""
    T, N, K = shape
    g = torch.Generator().manual_seed(T)
    for dtype in (BF, HF):
        x, w = sparse(T, K, g, dtype), sparse(N, K, g, dtype)
        pre, dy = (torch.randn(T, N, generator=g) * 2).to(dtype), torch.randn(T, N, generator=g).to(dtype)
        args = dict(act=act, pre=None if act == "none" else pre.cuda(), out_dtype=F32, need_db=True)
        dx, dw, db = bm.linear_backward(dy.cuda(), x.cuda(), w.cuda(), round_dz=True, **args)
        whole = bm.linear_backward(dy.cuda(), x.cuda(), w.cuda(), **args)
        assert torch.equal(db, whole[2])
        if act in ("none", "relu"):
            assert torch.equal(dx, whole[0]) and torch.equal(dw, whole[1])
        dy, x, w = dy.cuda().double(), x.cuda().double(), w.cuda().double()
        dz = dy * ex.act_slope(pre.cuda().double(), act)
        e = 2.0 ** -17 * dy.abs()
        e = e + ex.half_ulp(dtype) * (dz.abs() + e) + 2.0 ** -25 * (dtype == HF)
        m = dz.abs() + e
        for got, want, err, mag in ((dx, dz @ w, e @ w.abs(), m @ w.abs()),
                                    (dw, dz.t() @ x, e.t() @ x.abs(), m.t() @ x.abs())):
            assert over(got, want, err + ex.sum_bound(4) * mag + 2.0 ** -24 * want.abs()) <= 1


@pytest.mark.parametrize("T,K", [(1, 1), (40, 40), (300, 64), (1500, 1032)])
def test_gelu_of_negative_values(bm, T, K):
    """Relative to the value, down to where float32 ends: a sum of 1 and erf
    would leave nothing of it."""
    z = torch.arange(-13.0, -2.0, 1 / 64).to(HF)                                # (exact in float16)
    x, w = torch.zeros(T, K, dtype=HF), torch.zeros(z.numel(), K, dtype=HF)
    x[:, 0], w[:, 0] = 1, z
    z64 = z.double()
    # The argument z / sqrt 2 is off by 2^-23 of itself, twice its square, 169, times that in the result: 2^-15.6;
    # erfc's own error and the products' roundings, together below 2^-18.  A value below 2^-126 may be lost.
    y, _ = bm.linear(x.cuda(), w.cuda(), act="gelu", out_dtype=F32)
    want = ex.act(z64, "gelu").cuda()
    assert (want[-1] < -0.01) and (want < 0).all()
    worst = over(y, want, 2.0 ** -15.3 * want.abs() + 2.0 ** -126)
    say(f"[experts] gelu T={T}: largest error {worst:.2f} of its bound")
    assert worst <= 1
    # The slope's two terms, of opposite signs, the first at most a quarter of the second: 2^-15.6 / 4 of the first,
    # and of the second e^(-z^2 / 2) with an argument to 85, off by 2^-23 of itself in the square and again in the
    # exponential's base 2: 2^-15.6; both over the three quarters that are left.
    if T == 1:
        _, _, db = bm.linear_backward(torch.ones(1, z.numel(), dtype=HF, device="cuda"), x.cuda(), w.cuda(), act="gelu",
                                      pre=z.cuda()[None], need_dx=False, need_dw=False, need_db=True, out_dtype=F32)
        want = ex.act_slope(z64, "gelu").cuda()
        worst = over(db, want, 2.0 ** -14.8 * want.abs() + 2.0 ** -124)
        say(f"[experts] gelu's slope: largest error {worst:.2f} of its bound")
        assert worst <= 1


@pytest.mark.parametrize("round_dz", [False, True])
def test_linear_backward_captured_and_replayed(bm, round_dz):
    """Two graphs of one call, with a workspace each from their own pools."""
    T, N, K = 600, 264, 520
    g = torch.Generator(device="cuda").manual_seed(3)
    make = lambda *s: torch.empty(*s, dtype=BF, device="cuda").normal_(generator=g)  # noqa: E731
    dy, x, w, pre = make(T, N), make(T, K), make(N, K), make(T, N)

    def run():
        return bm.linear_backward(dy, x, w, act="gelu", pre=pre, need_db=True, round_dz=round_dz)
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, run()))
    for _ in range(4):
        for t in (dy, x, w, pre):
            t.normal_(generator=g)
        for graph, _ in graphs:
            graph.replay()
        want = run()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("R,N,K,pad", [(300, 72, 136, 0), (2048, 72, 72, 0), (300, 33, 17, 1), (3000, 264, 1032, 0)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_weights_gradient_added_to_16_bits(bm, R, N, K, pad, dtype):
    """accumulate into the operands' type: the sum in float32, rounded once."""
    g = torch.Generator().manual_seed(R + N)
    dy, x = padded(torch.randn(R, N, generator=g).to(dtype), pad, 0), padded(torch.randn(R, K, generator=g).to(dtype), pad, 0)
    was = (torch.randn(2, N, K, generator=g) * 30).to(dtype)
    dw = was.cuda()
    off = torch.tensor([0, R - 100, R], dtype=torch.int32).cuda()
    assert bm.expert_matmul_dw(dy, x, off, dw=dw, accumulate=True) is dw
    for e, s in ((0, slice(0, R - 100)), (1, slice(R - 100, R))):
        d, v = dy[s].double(), x[s].double()
        want, mag = was[e].cuda().double() + d.t() @ v, d.abs().t() @ v.abs()
        assert over(dw[e], want, ex.half_ulp(dtype) * want.abs() + 1.01 * ex.sum_bound(R) * mag + 2.0 ** -22 *
                    (want.abs() + was[e].cuda().double().abs()) + 2.0 ** -25 * (dtype == HF)) <= 1
