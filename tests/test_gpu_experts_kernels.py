"""Every kernel of the 16-bit products against float64, per element, in both
types (_experts_cases.py: which sizes take which kernel): through row maps and
without, into the operands' type and float32, and the same bits twice."""
import pytest

import _experts as ex
import _experts_cases as cases
from _gpu import require_gpu, say, torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def ident(case):
    return f"{case[0]} E{len(case[1])} R{sum(case[1])} N{case[2]} K{case[3]}".replace(" ", "_")


def random(g, place, *shape, dtype):
    """A dense tensor whose first element lies `place` behind an aligned
    address."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.empty(n + place + 8, dtype=dtype, device="cuda").normal_(generator=g)
    return buf[place:place + n].view(shape)


def inputs(case, dtype):
    _, counts, N, K, place = case
    g = torch.Generator(device="cuda").manual_seed(N * 7 + K)
    R, E = sum(counts), len(counts)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    make = lambda *s: random(g, place, *s, dtype=dtype)  # noqa: E731
    perm = torch.randperm(R, generator=torch.Generator().manual_seed(R)).to(torch.int32).cuda()
    say(f"[experts] {ident(case)} {dtype}")
    return make, R, E, N, K, off, perm


def groups(counts):
    at = 0
    for e, n in enumerate(counts):
        if n:
            yield e, slice(at, at + n)
        at += n


def within(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() / (bound + 1e-300)).max().item()
    assert worst <= 1, (what, worst)


def check_rows(case, dtype, call, n_in, n_out, product):
    """call(a, w, offsets, a map, output map, out_dtype) and product(rows, W):
    a group's rows in float64."""
    make, R, E, N, K, off, perm = inputs(case, dtype)
    a, w = make(R, n_in), make(E, N, K)
    y = call(a, w, off, None, perm, None)                     # row r to perm[r]
    y32 = call(a, w, off, perm, None, F32)                    # row r is perm[r]
    assert torch.equal(y, call(a, w, off, None, perm, None)) and torch.equal(y32, call(a, w, off, perm, None, F32))
    assert y.dtype == dtype and y32.dtype == F32 and y.shape == (R, n_out)
    p = perm.long()
    for e, s in groups(case[1]):
        we = w[e].double()
        for got, rows, u in ((y[p[s]], a[s], ex.half_ulp(dtype)), (y32[s], a[p[s]], 2.0 ** -24)):
            rows = rows.double()
            want, mag = product(rows, we), product(rows.abs(), we.abs())
            # (fp16 is left at 2^-25 below its smallest normal value)
            within(got, want, u * want.abs() + ex.sum_bound(n_in) * mag + 2.0 ** -25 * (got.dtype == HF), (ident(case), e))


@TYPES
@pytest.mark.parametrize("case", cases.FORWARD, ids=ident)
def test_forward(bm, case, dtype):
    _, _, N, K, _ = case
    check_rows(case, dtype, lambda x, w, off, xr, yr, dt: bm.expert_matmul(x, w, off, x_rows=xr, y_rows=yr, out_dtype=dt),
               K, N, lambda rows, w: rows @ w.t())


@TYPES
@pytest.mark.parametrize("case", cases.DX, ids=ident)
def test_rows_gradient(bm, case, dtype):
    _, _, N, K, _ = case
    check_rows(case, dtype,
               lambda dy, w, off, dyr, dxr, dt: bm.expert_matmul_dx(dy, w, off, dy_rows=dyr, dx_rows=dxr, out_dtype=dt),
               N, K, lambda rows, w: rows @ w)


@TYPES
@pytest.mark.parametrize("maps", ["", "x", "dy", "both"])
@pytest.mark.parametrize("case", cases.DW, ids=ident)
def test_weights_gradient(bm, case, dtype, maps):
    make, R, E, N, K, off, perm = inputs(case, dtype)
    dy, x = make(R, N), make(R, K)
    other = perm.flip(0).contiguous()
    kw = {"dy_rows": perm} if maps == "dy" else {"x_rows": perm} if maps == "x" else \
        {"dy_rows": perm, "x_rows": other} if maps else {}
    dw = bm.expert_matmul_dw(dy, x, off, **kw)
    assert torch.equal(dw, bm.expert_matmul_dw(dy, x, off, **kw))
    acc = random(torch.Generator(device="cuda").manual_seed(1), 0, E, N, K, dtype=F32)
    was = acc.clone()
    bm.expert_matmul_dw(dy, x, off, dw=acc, accumulate=True, **kw)
    dyg = dy[perm.long()] if "dy_rows" in kw else dy
    xg = x[kw["x_rows"].long()] if "x_rows" in kw else x
    seen = set()
    for e, s in groups(case[1]):
        seen.add(e)
        d, v = dyg[s].double(), xg[s].double()
        want, mag = d.t() @ v, d.abs().t() @ v.abs()
        b = ex.sum_bound(s.stop - s.start) * mag
        within(dw[e], want, ex.half_ulp(dtype) * want.abs() + b + 2.0 ** -25 * (dtype == HF), (ident(case), e))
        sums = was[e].double() + want                        # one more addition, one more rounding
        within(acc[e], sums, b + 2.0 ** -23 * (sums.abs() + was[e].double().abs()), (ident(case), e, "accumulated"))
    for e in set(range(E)) - seen:
        assert (dw[e] == 0).all() and torch.equal(acc[e], was[e])


@pytest.mark.parametrize("R,N,K", [(5, 64, 72), (300, 33, 17), (1, 2056, 264), (4000, 264, 512)])
def test_maps_over_a_matrix_without_rows(bm, R, N, K):
    E = 1 if R < 300 else 3
    off = torch.tensor([0] + [R] * E, dtype=torch.int32).cuda()
    w = torch.randn(E, N, K, device="cuda").to(BF)
    rows = torch.arange(R, dtype=torch.int32, device="cuda")
    none = lambda n: torch.empty(0, n, dtype=BF, device="cuda")  # noqa: E731
    x, dy = torch.randn(R, K, device="cuda").to(BF), torch.randn(R, N, device="cuda").to(BF)
    assert (bm.expert_matmul(none(K), w, off, x_rows=rows) == 0).all()
    assert (bm.expert_matmul_dx(none(N), w, off, dy_rows=rows) == 0).all()
    assert (bm.expert_matmul_dw(dy, none(K), off, x_rows=rows) == 0).all()
    assert (bm.expert_matmul_dw(none(N), x, off, dy_rows=rows) == 0).all()
    assert bm.expert_matmul(x, w, off, y_rows=rows, y=none(N)).shape == (0, N)
    assert bm.expert_matmul_dx(dy, w, off, dx_rows=rows, dx=none(K)).shape == (0, K)
    torch.cuda.synchronize()
