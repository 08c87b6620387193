"""Every kernel of the products in 8 bits against exact sums, per element
(_rows8_cases.py: which sizes take which kernel): through row maps and without, into
each type, and the same bits twice."""
import pytest

import _rows8 as r8
import _rows8_cases as cases
from _gpu import require_gpu, say, torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def ident(case):
    return f"{case[0]} E{len(case[1])} R{sum(case[1])} N{case[2]} K{case[3]} at{case[4]}".replace(" ", "_")


def random(g, place, *shape):
    n = 1
    for s in shape:
        n *= s
    buf = torch.randint(-127, 128, (n + place + 16,), dtype=torch.int8, device="cuda", generator=g)
    return buf[place:place + n].view(shape)


@pytest.mark.parametrize("case", cases.I8, ids=ident)
def test_every_kernel(bm, case):
    _, counts, N, K, place = case
    g = torch.Generator(device="cuda").manual_seed(N * 7 + K)
    R, E = sum(counts), len(counts)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    say(f"[i8] {ident(case)}")
    x, w = random(g, place, R, K), random(g, place, E, N, K)
    xs = torch.rand(R, device="cuda", generator=g) + 0.1
    ws = torch.rand(E, N, device="cuda", generator=g) * 1e-4 + 1e-5
    # exact: sums below 2^31 in float64, on the device, a group at a time
    want = torch.empty(R, N, dtype=torch.float64, device="cuda")
    at = 0
    for e, n in enumerate(counts):
        if n:
            want[at:at + n] = x[at:at + n].double() @ w[e].double().t() * xs[at:at + n, None].double() * ws[e].double()
        at += n
    q, v = bm.Rows8(x, xs), bm.Rows8(w, ws)
    perm = torch.randperm(R, generator=torch.Generator().manual_seed(R)).to(torch.int32).cuda()

    def near(got, want, what):
        bound = r8.product_bound(want, got.dtype)
        worst = ((got.double() - want).abs() / (bound + 1e-30)).max().item()
        say(f"[i8] {what} {got.dtype}: largest error {worst:.2f} of its bound")
        assert worst <= 1, what
    for dtype in (BF, HF, F32):
        y = bm.expert_matmul_i8(q, v, off, out_dtype=dtype)
        near(y, want, "plain")
        assert torch.equal(y, bm.expert_matmul_i8(q, v, off, out_dtype=dtype))
    # rows gathered and scattered: call row r is x row perm[r], and goes to y row perm[r]
    gathered = torch.empty_like(want)
    at = 0
    for e, n in enumerate(counts):
        if n:
            i = perm[at:at + n].long()
            gathered[i] = x[i].double() @ w[e].double().t() * xs[i, None].double() * ws[e].double()
        at += n
    near(bm.expert_matmul_i8(q, v, off, x_rows=perm, y_rows=perm), gathered, "mapped")
