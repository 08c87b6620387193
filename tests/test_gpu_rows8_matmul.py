"""Products grouped by expert in 8 bits against exact sums in float64.  Bound:
_rows8.product_bound (the sum is exact; its way to float32, two products and the
output's rounding are not)."""
import pytest

import _experts as ex
import _rows8 as r8
from _gpu import require_gpu, say, torch
from test_gpu_experts import BF, F32, GROUPS, HF, check, gen, offsets_of, place

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def codes(g, *shape, pad=0, shift=0):
    """Random codes on the device, rows `pad` bytes apart from an address `shift`
    off, and their values."""
    v = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    return place(v, pad, shift, hold=99), v.double()


def weights(bm, g, E, N, K, pad=0, shift=0):
    q, v = codes(g, E, N, K, pad=pad, shift=shift)
    s = torch.rand(E, N, generator=g) * 0.01 + 1e-4
    return bm.Rows8(q, s.cuda()), v, s.double()


def rows(bm, g, R, K, pad=0, shift=0):
    q, v = codes(g, R, K, pad=pad, shift=shift)
    s = torch.rand(R, generator=g) * 0.02 + 1e-3
    return bm.Rows8(q, s.cuda()), v, s.double()


# N, K, bytes between rows, first byte's place: whole 16-byte pieces, odd sizes, strides and addresses
SHAPES = [(128, 128, 0, 0), (256, 512, 0, 0), (1, 1, 0, 0), (17, 33, 0, 0), (200, 208, 16, 16), (96, 144, 3, 1),
          (264, 1040, 0, 0), (130, 7, 1, 0), (512, 2048, 0, 0), (130, 144, 0, 0), (7, 2192, 0, 0), (1, 128, 0, 0),
          (72, 130, 0, 2), (300, 1001, 0, 0), (136, 272, 2, 4)]


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_expert_matmul_i8(bm, groups, shape):
    N, K, pad, shift = shape
    counts, behind = GROUPS[groups]
    E, n = len(counts), sum(counts)
    R = n + behind
    g = gen(1000 * N + K)
    x, x64, xs = rows(bm, g, max(R, 1), K, pad, shift)
    x.scale[n:] = float("nan")                                   # rows of no group are not read
    w, w64, ws = weights(bm, g, E, N, K, pad, shift)
    off = offsets_of(counts)
    say(f"[i8] {groups} N={N} K={K} pad={pad} shift={shift}")
    want = r8.expert_rows(x64[:n], xs[:n], w64, ws, off)
    for dtype in (BF, HF, F32):
        y = place(torch.full((max(R, 1), N), 7.0, dtype=dtype), pad, shift, hold=5.0)
        bm.expert_matmul_i8(x, w, off.cuda(), y=y)
        check(y[:n], want, r8.product_bound(want, dtype), f"i8 {groups} {shape} {dtype}")
        assert (y[n:] == 7).all()                                # nor written
        if pad and R > 1:
            assert (y.as_strided((R - 1, pad), (N + pad, 1), shift + N) == 5).all()


@pytest.mark.parametrize("T,k,E,N,K", [(5, 2, 8, 128, 128), (37, 8, 16, 200, 528), (1, 8, 64, 256, 1024), (1, 8, 64, 250, 1001),
                                       (200, 3, 4, 65, 39), (16, 4, 256, 64, 1024)])
def test_maps_gather_and_scatter(bm, T, k, E, N, K):
    """bucket's perm as the maps; entries outside the matrices read as codes and
    scale 0 and are not written."""
    g = gen(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    x, x64, xs = rows(bm, g, T, K)
    w, w64, ws = weights(bm, g, E, N, K)
    _, off, perm, _, _ = bm.bucket(ids.cuda(), E)
    p = perm.cpu()
    say(f"[i8] maps T={T} k={k} E={E} N={N} K={K}")
    src = torch.div(p.long(), k, rounding_mode="floor")
    got = r8.expert_rows(x64[src], xs[src], w64, ws, off.cpu())
    want = torch.empty_like(got)
    want[p.long()] = got
    y = bm.expert_matmul_i8(x, w, off, x_rows=perm, x_div=k, y_rows=perm)
    check(y, want, r8.product_bound(want, BF), "gather, scatter")
    bad = p.clone()
    bad[::3] = -1
    bad[1::5] = T * k + 100
    bad[0] = 2 ** 31 - 1
    out = torch.full((T * k, N), 7.0, dtype=F32, device="cuda")
    bm.expert_matmul_i8(x, w, off, x_rows=bad.cuda(), x_div=k, y_rows=perm, y=out)
    at = torch.div(bad.long(), k, rounding_mode="floor")
    ok = (bad >= 0) & (at < T)
    at[~ok] = 0
    got = r8.expert_rows(x64[at], xs[at] * ok, w64, ws, off.cpu())
    want[p.long()] = got
    check(out, want, r8.product_bound(want, F32), "rows of x that are not there")
    out.fill_(7.0)
    bm.expert_matmul_i8(x, w, off, x_rows=perm, x_div=k, y_rows=bad.cuda(), y=out)
    got = r8.expert_rows(x64[src], xs[src], w64, ws, off.cpu())
    want.fill_(7.0)
    there = (bad >= 0) & (bad < T * k)
    want[bad[there].long()] = got[there]
    check(out, want, r8.product_bound(want, F32), "rows of y that are not there")
    # a share of the experts: the others' pairs are 0
    e0, e1 = E // 4, E // 4 + max(E // 2, 1)
    part = bm.Rows8(w.codes[e0:e1], w.scale[e0:e1])
    y = bm.expert_matmul_i8(x, part, off[e0:e1 + 1], x_rows=perm, x_div=k, y_rows=perm, out_dtype=F32)
    lo, hi = int(off[e0]), int(off[e1])
    want.zero_()
    want[p[lo:hi].long()] = got[lo:hi]
    check(y, want, r8.product_bound(want, F32), "a share")


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 300, 2048), (5, 520, 4096), (64, 136, 4112), (300, 1000, 2000), (129, 257, 513),
                                   (2048, 264, 1024), (16, 2056, 7168), (1, 4096, 7167), (700, 512, 130)])
def test_dense(bm, T, N, K):
    """Without offsets: one product of all rows, weights [N, K]."""
    g = gen(T + N)
    x, x64, xs = rows(bm, g, T, K)
    w, w64, ws = weights(bm, g, 1, N, K)
    want = r8.expert_rows(x64, xs, w64, ws, [0, T])
    say(f"[i8] dense T={T} N={N} K={K}")
    for dtype in (BF, F32):
        y = bm.expert_matmul_i8(x, bm.Rows8(w.codes[0], w.scale[0]), out_dtype=dtype)
        check(y, want, r8.product_bound(want, dtype), f"dense {dtype}")
    # a view's columns and rows, every second scale
    if T > 2 and K > 64:
        part = bm.Rows8(x.codes[::2, 16:], x.scale[::2])
        y = bm.expert_matmul_i8(part, bm.Rows8(w.codes[0, :, 16:], w.scale[0]), out_dtype=F32)
        want = r8.expert_rows(x64[::2, 16:], xs[::2], w64[:, :, 16:], ws, [0, (T + 1) // 2])
        check(y, want, r8.product_bound(want, F32), "views")


@pytest.mark.parametrize("K", [65536 + 48, (1 << 17) - 1])
def test_sums_at_the_edge_of_int32(bm, K):
    """All codes -128 (which no quantisation gives) or 127 at long K: the largest
    sums."""
    for T, N in ((3, 40), (200, 200)):
        x = torch.full((T, K), -128, dtype=torch.int8)
        w = torch.full((N, K), -128, dtype=torch.int8)
        x[1::3], w[1::2] = 127, 127
        say(f"[i8] largest sums K={K} T={T} N={N}")
        one = torch.ones(max(T, N))
        y = bm.expert_matmul_i8(bm.Rows8(x.cuda(), one[:T].cuda()), bm.Rows8(w.cuda(), one[:N].cuda()), out_dtype=F32)
        want = x.double() @ w.double().t()
        check(y, want, r8.product_bound(want, F32), "largest sums")


def test_scales_that_are_not_finite(bm):
    """A row whose scale is NaN (its activations were) is NaN, no other is."""
    g = gen(8)
    x = torch.randn(40, 256, generator=g).to(BF)
    x[7, 3], x[9, 200] = float("inf"), float("nan")
    w = bm.quantize_rows(torch.randn(64, 256, generator=g).cuda())
    y = bm.expert_matmul_i8(bm.quantize_rows(x.cuda()), w, out_dtype=F32).cpu()
    bad = torch.zeros(40, dtype=torch.bool)
    bad[[7, 9]] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def test_no_rows(bm):
    w, _, _ = weights(bm, gen(1), 3, 16, 32)
    x = bm.Rows8(torch.empty(0, 32, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert bm.expert_matmul_i8(x, w, off).shape == (0, 16)
    # a map over a matrix without rows: all rows read as zeros
    y = bm.expert_matmul_i8(x, w, torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda"),
                            x_rows=torch.arange(5, dtype=torch.int32, device="cuda"), out_dtype=F32)
    assert (y == 0).all()
