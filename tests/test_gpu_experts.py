"""The 16-bit expert layer's operators against their formulas in float64, at
the sizes, strides and masks where they can go wrong.  Every comparison is per
element against a bound derived from the arithmetic: one rounding of the
result (half_ulp), fp32 sums (sum_bound times the sum of absolute values) and,
where an operand is rounded on the way, that rounding's share."""
import pytest

import _experts as ex
from _gpu import require_gpu, say, torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TINY = 1e-30


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=BF, scale=1.0, pad=0, shift=0, hold=float("nan")):
    """A device tensor whose rows lie `pad` elements further apart than they
    are long and begin `shift` elements behind an aligned address, with
    `hold` in between, and its values in float64."""
    v = (torch.randn(*shape, generator=g) * scale).to(dtype)
    return place(v, pad, shift, hold), v.double()


def place(v, pad=0, shift=0, hold=float("nan")):
    ld = v.shape[-1] + pad
    n = v.numel() // max(v.shape[-1], 1)
    buf = torch.full((shift + n * ld + 8,), hold, dtype=v.dtype, device="cuda")
    strides = [ld * (n // max(v.shape[0], 1)) if v.dim() == 3 else ld] + ([ld] if v.dim() == 3 else []) + [1]
    t = buf.as_strided(v.shape, strides, shift)
    t.copy_(v)
    return t


def check(got, want, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == want.shape
    assert torch.isfinite(g).all(), f"{what}: not finite"
    over = ((g - want).abs() - bound).max().item() if g.numel() else 0.0
    worst = ((g - want).abs() / (bound + TINY)).max().item() if g.numel() else 0.0
    say(f"[experts] {what}: largest error {worst:.2f} of its bound")
    assert over <= 0, f"{what}: over its bound by {over:.3e} ({worst:.2f} times)"


def offsets_of(counts):
    return torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(torch.int32)


# counts (an expert without rows, one row, a row over a tile...), rows behind the last group
GROUPS = {
    "one": ([1], 0),
    "empty": ([0, 0, 0], 3),
    "mixed": ([0, 1, 7, 0, 129, 64, 3], 5),
    "even": ([64, 64, 64, 64], 0),
    "long": ([300, 0, 515], 1),
    "many": ([i % 4 for i in range(300)], 2),
    "decode": ([1 if i % 5 == 0 else 0 for i in range(70)], 0),
    "pairs": ([2, 0, 16, 17, 0, 5, 33], 0),
}
# N, K, padding between rows, first element's place: rows on 16 bytes, odd sizes, odd strides, odd addresses
SHAPES = [(128, 64, 0, 0), (256, 256, 0, 0), (1, 1, 0, 0), (17, 33, 0, 0), (200, 104, 8, 8), (96, 72, 3, 1),
          (264, 520, 0, 0), (130, 7, 1, 0), (512, 1024, 0, 0), (130, 72, 0, 0), (7, 1096, 0, 0), (1, 64, 0, 0)]


def experts_case(groups, N, K, dtype, pad, shift, seed=0):
    counts, behind = GROUPS[groups]
    E, n = len(counts), sum(counts)
    R = n + behind
    g = gen(seed + 1000 * N + K)
    return E, n, R, offsets_of(counts), g


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_expert_matmul(bm, groups, shape):
    N, K, pad, shift = shape
    dtype = HF if (N + K) % 16 else BF
    E, n, R, off, g = experts_case(groups, N, K, dtype, pad, shift)
    x, x64 = rnd(g, max(R, 1), K, dtype=dtype, pad=pad, shift=shift)
    if R > n:
        x[n:] = float("nan")                                     # rows of no group are not read
    w, w64 = rnd(g, E, N, K, dtype=dtype, pad=pad, shift=shift)
    say(f"[experts] matmul {groups} N={N} K={K} pad={pad} shift={shift} {dtype}")
    y = place(torch.full((max(R, 1), N), 7.0, dtype=dtype), pad, shift, hold=5.0)
    bm.expert_matmul(x, w, off.cuda(), y=y)
    want, mag = ex.expert_rows(x64[:n], w64, off)
    check(y[:n], want, ex.half_ulp(dtype) * want.abs() + ex.sum_bound(K) * mag + 2.0 ** -24 * (dtype == HF),
          f"matmul {groups} {shape}")
    assert (y[n:] == 7).all()                                    # nor written
    if pad and R > 1:
        assert (y.as_strided((R - 1, pad), (N + pad, 1), shift + N) == 5).all()
    y32 = bm.expert_matmul(x, w, off.cuda(), out_dtype=F32)
    check(y32[:n], want, 2.0 ** -24 * want.abs() + ex.sum_bound(K) * mag, f"matmul {groups} {shape} fp32")


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_expert_matmul_dx(bm, groups, shape):
    N, K, pad, shift = shape
    dtype = BF if (N + K) % 16 else HF
    E, n, R, off, g = experts_case(groups, N, K, dtype, pad, shift, 1)
    dy, dy64 = rnd(g, max(R, 1), N, dtype=dtype, pad=pad, shift=shift)
    if R > n:
        dy[n:] = float("nan")
    w, w64 = rnd(g, E, N, K, dtype=dtype, pad=pad, shift=shift)
    say(f"[experts] dx {groups} N={N} K={K} pad={pad} shift={shift} {dtype}")
    dx = place(torch.full((max(R, 1), K), 7.0, dtype=dtype), pad, shift)
    bm.expert_matmul_dx(dy, w, off.cuda(), dx=dx)
    want, mag = ex.expert_rows(dy64[:n], w64, off, transposed=True)
    check(dx[:n], want, ex.half_ulp(dtype) * want.abs() + ex.sum_bound(N) * mag + 2.0 ** -24 * (dtype == HF),
          f"dx {groups} {shape}")
    assert (dx[n:] == 7).all()


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_expert_matmul_dw(bm, groups, shape):
    N, K, pad, shift = shape
    dtype = HF if (N + K) % 16 else BF
    E, n, R, off, g = experts_case(groups, N, K, dtype, pad, shift, 2)
    dy, dy64 = rnd(g, max(R, 1), N, dtype=dtype, pad=pad, shift=shift)
    x, x64 = rnd(g, max(R, 1), K, dtype=dtype, pad=pad, shift=shift)
    if R > n:
        dy[n:] = float("nan")
        x[n:] = float("nan")
    say(f"[experts] dw {groups} N={N} K={K} pad={pad} shift={shift} {dtype}")
    dw = place(torch.full((E, N, K), float("nan"), dtype=dtype), pad, shift)
    bm.expert_matmul_dw(dy, x, off.cuda(), dw=dw)
    want, mag = ex.expert_dw(dy64[:n], x64[:n], off)
    rows = max(GROUPS[groups][0])
    check(dw, want, ex.half_ulp(dtype) * want.abs() + ex.sum_bound(rows) * mag + 2.0 ** -24 * (dtype == HF),
          f"dw {groups} {shape}")
    # added to what is there, in fp32: one more addition's rounding
    acc, a64 = rnd(g, E, N, K, dtype=F32)
    bm.expert_matmul_dw(dy, x, off.cuda(), dw=acc, accumulate=True)
    check(acc, a64 + want, 2.0 ** -24 * (a64 + want).abs() + ex.sum_bound(rows) * mag + 2.0 ** -23 * a64.abs(),
          f"dw {groups} {shape} accumulated")


@pytest.mark.parametrize("T,k,E,N,K", [(5, 2, 8, 128, 64), (37, 8, 16, 200, 264), (1, 8, 64, 256, 512),
                                       (200, 3, 4, 65, 39), (16, 4, 256, 64, 1024)])
def test_maps_gather_and_scatter(bm, T, k, E, N, K):
    """bucket's perm as the maps: tokens gathered, rows back in pair order;
    entries outside the matrices read zeros and are not written."""
    g = gen(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    x, x64 = rnd(g, T, K)
    w, w64 = rnd(g, E, N, K)
    counts, off, perm, _, _ = bm.bucket(ids.cuda(), E)
    p = perm.cpu()
    say(f"[experts] maps T={T} k={k} E={E} N={N} K={K}")
    y = bm.expert_matmul(x, w, off, x_rows=perm, x_div=k, y_rows=perm)
    rows, mag = ex.expert_rows(ex.mapped(x64, p, k), w64, off.cpu())
    want, wmag = torch.empty_like(rows), torch.empty_like(mag)
    want[p.long()], wmag[p.long()] = rows, mag
    check(y, want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(K) * wmag, "gather, scatter")
    dy, dy64 = rnd(g, T * k, N)
    dx = bm.expert_matmul_dx(dy, w, off, dy_rows=perm, dx_rows=perm)
    rows, mag = ex.expert_rows(ex.mapped(dy64, p), w64, off.cpu(), transposed=True)
    want, wmag = torch.empty_like(rows), torch.empty_like(mag)
    want[p.long()], wmag[p.long()] = rows, mag
    check(dx, want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(N) * wmag, "dx gather, scatter")
    dw = bm.expert_matmul_dw(dy, x, off, dy_rows=perm, x_rows=perm, x_div=k)
    want, mag = ex.expert_dw(ex.mapped(dy64, p), ex.mapped(x64, p, k), off.cpu())
    check(dw, want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(T) * mag, "dw gathered")
    # entries outside
    bad = p.clone()
    bad[::3] = -1
    bad[1::5] = T * k + 100
    bad[0] = 2 ** 31 - 1
    out = torch.full((T * k, N), 7.0, dtype=BF, device="cuda")
    bm.expert_matmul(x, w, off, x_rows=bad.cuda(), x_div=k, y_rows=bad.cuda(), y=out)
    ok = (bad >= 0) & (bad < T * k)
    rows, mag = ex.expert_rows(ex.mapped(x64, bad, k), w64, off.cpu())
    want = torch.full((T * k, N), 7.0, dtype=ex.F64)
    bound = torch.zeros_like(want)
    at = bad[ok].long()
    want[at] = rows[ok]
    bound[at] = ex.half_ulp(BF) * rows[ok].abs() + ex.sum_bound(K) * mag[ok]
    check(out, want, bound, "entries outside")
    dw = bm.expert_matmul_dw(dy, x, off, dy_rows=bad.cuda(), x_rows=bad.cuda(), x_div=k)
    want, mag = ex.expert_dw(ex.mapped(dy64, bad), ex.mapped(x64, bad, k), off.cpu())
    check(dw, want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(T) * mag, "dw, entries outside")


def compare(got, want, bound, what):
    """check() where the operands are large: the oracle's products in float64
    on the GPU."""
    assert torch.isfinite(got).all(), what
    d = (got.double() - want).abs()
    worst = (d / (bound + TINY)).max().item()
    say(f"[experts] {what}: largest error {worst:.2f} of its bound")
    assert worst <= 1, what


def large(g, *shape, dtype=BF, scale=1.0):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0, scale, generator=g)


# (E, rows of the groups, N, K): more tiles than compute units, of every size and an uneven end; few tiles and a
# long contraction, which is split
MANY = [(1, [5000], 2840, 200), (3, [4100, 0, 2000], 1992, 328), (40, [150, 3, 90, 400] * 10, 1160, 456),
        (300, [37] * 300, 392, 264), (1, [8192], 2816, 72)]
SPLIT = [(1, [64], 128, 4096), (1, [300], 200, 7168), (4, [5, 0, 17, 2], 136, 4104), (1, [1], 8, 6144),
         (2, [130, 257], 257, 2056)]


@pytest.mark.parametrize("case", MANY + SPLIT, ids=lambda c: f"E{c[0]}R{sum(c[1])}N{c[2]}K{c[3]}")
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_many_tiles_and_split_contractions(bm, case, dtype):
    E, counts, N, K = case
    g = torch.Generator(device="cuda").manual_seed(N + K)
    off = offsets_of(counts)
    R = int(off[-1])
    if case in SPLIT:
        assert bm.expert_matmul_workspace_bytes(bm.MATMUL_DX, E, R, K, N) > 0 or R < 65
    x, w, dy = large(g, R, K, dtype=dtype), large(g, E, N, K, dtype=dtype), large(g, R, N, dtype=dtype)
    perm = torch.randperm(R, generator=gen(1)).to(torch.int32).cuda()
    say(f"[experts] E={E} R={R} N={N} K={K} {dtype}")
    offc = off.cuda()
    y, y32 = bm.expert_matmul(x, w, offc, y_rows=perm), bm.expert_matmul(x, w, offc, x_rows=perm, out_dtype=F32)
    dx = bm.expert_matmul_dx(dy, w, offc, dy_rows=perm)
    dw = bm.expert_matmul_dw(dy, x, offc, dy_rows=perm)
    dw2 = bm.expert_matmul_dw(dy, x, offc, out_dtype=F32)
    for a, f in ((y, lambda: bm.expert_matmul(x, w, offc, y_rows=perm)),
                 (dw, lambda: bm.expert_matmul_dw(dy, x, offc, dy_rows=perm))):
        assert torch.equal(a, f())                                      # the same bits again
    u, small = ex.half_ulp(dtype), 2.0 ** -24 * (dtype == HF)
    p = perm.long()
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        wd, xs, dys = w[e].double(), x[s].double(), dy[p[s]].double()
        want, mag = xs @ wd.t(), xs.abs() @ wd.abs().t()
        if s.stop > s.start:
            compare(y[p[s]], want, u * want.abs() + ex.sum_bound(K) * mag + small, f"y of expert {e}")
            xg = x[p[s]].double()
            want, mag = xg @ wd.t(), xg.abs() @ wd.abs().t()
            compare(y32[s], want, 2.0 ** -24 * want.abs() + ex.sum_bound(K) * mag, f"y32 of expert {e}")
            want, mag = dys @ wd, dys.abs() @ wd.abs()
            compare(dx[s], want, u * want.abs() + ex.sum_bound(N) * mag + small, f"dx of expert {e}")
        n = s.stop - s.start
        want, mag = dys.t() @ xs, dys.t().abs() @ xs.abs()
        compare(dw[e], want, u * want.abs() + ex.sum_bound(n) * mag + small, f"dw of expert {e}")
        dys = dy[s].double()
        want, mag = dys.t() @ xs, dys.t().abs() @ xs.abs()
        compare(dw2[e], want, 2.0 ** -24 * want.abs() + ex.sum_bound(n) * mag, f"dw32 of expert {e}")


@pytest.mark.parametrize("N,K,R", [(128, 128, 8192), (72, 264, 4000), (17, 33, 3000)])
def test_weights_gradient_split_over_rows(bm, N, K, R):
    g = torch.Generator(device="cuda").manual_seed(R)
    assert bm.expert_matmul_workspace_bytes(bm.MATMUL_DW, 2, R, N, K) >= 8 * 2 * N * K
    dy, x = large(g, R, N), large(g, R, K)
    off = offsets_of([R - 700, 500])                                    # 200 rows behind the last group
    dy[R - 200:] = float("nan")
    x[R - 200:] = float("nan")
    perm = torch.arange(R - 1, -1, -1, dtype=torch.int32)
    acc = large(g, 2, N, K, dtype=F32)
    a64 = acc.double()
    dw = bm.expert_matmul_dw(dy, x, off.cuda())
    bm.expert_matmul_dw(dy, x, off.cuda(), dw=acc, accumulate=True)
    dwm = bm.expert_matmul_dw(dy, x.flip(0), off.cuda(), x_rows=perm.cuda())
    for e, s in ((0, slice(0, R - 700)), (1, slice(R - 700, R - 200))):
        want, mag = dy[s].double().t() @ x[s].double(), dy[s].double().abs().t() @ x[s].double().abs()
        bound = ex.half_ulp(BF) * want.abs() + ex.sum_bound(R) * mag
        compare(dw[e], want, bound, f"dw {e}")
        compare(dwm[e], want, bound, f"dw {e}, mapped")
        compare(acc[e], a64[e] + want, 2.0 ** -23 * ((a64[e] + want).abs() + a64[e].abs()) + ex.sum_bound(R) * mag,
                f"dw {e}, accumulated")


@pytest.mark.parametrize("N,K,pad", [(256, 512, 0), (72, 40, 0), (33, 17, 1)])
@pytest.mark.parametrize("side", ["dy", "x"])
def test_weights_gradient_leaves_out_what_a_map_takes(bm, N, K, pad, side):
    """A row that one operand's map takes adds nothing, though the other
    operand's row holds infinities and NaN."""
    R = 300
    g = gen(N + K)
    dy, dy64 = rnd(g, R, N, pad=pad)
    x, x64 = rnd(g, R, K, pad=pad)
    gone = torch.randperm(R, generator=g)[:90]
    gone = torch.cat([gone, torch.arange(128, 192)])                    # a whole stage of the contraction among them
    rows = torch.arange(R, dtype=torch.int32)
    rows[gone] = torch.where(gone % 2 == 0, -1, R + 5).to(torch.int32)
    hidden, h64 = (x, x64) if side == "dy" else (dy, dy64)
    hidden[gone.cuda()] = torch.tensor([float("nan"), float("inf")], dtype=BF, device="cuda")[(gone % 2).cuda()][:, None]
    h64[gone] = 0
    off = offsets_of([100, 0, 190])
    dw = bm.expert_matmul_dw(dy, x, off.cuda(), **{side + "_rows": rows.cuda()})
    want, mag = ex.expert_dw(dy64, x64, off)
    check(dw, want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(R) * mag, f"dw without {side}'s rows, N={N} K={K}")


@pytest.mark.parametrize("mapped", [False, True], ids=["contiguous", "mapped"])
def test_operands_beyond_4_gib(bm, mapped):
    """Rows and outputs more than 2^32 bytes from their matrix's beginning."""
    g = torch.Generator(device="cuda").manual_seed(5)
    K, N, rows = 7168, 136, 330000                                      # x: 4.7 GB
    x = torch.empty(rows, K, dtype=BF, device="cuda")
    n = 300
    at = torch.cat([torch.arange(5), torch.arange(rows - n + 5, rows)])
    x[at.cuda()] = large(g, n, K)
    w, dy = large(g, 2, N, K, scale=K ** -0.5), large(g, n, N)
    xs = x[at.cuda()].double()
    if mapped:
        m = at.to(torch.int32).cuda()
        off = offsets_of([100, 200]).cuda()
        y = bm.expert_matmul(x, w, off, x_rows=m)
        out = torch.zeros(rows, K, dtype=BF, device="cuda")
        bm.expert_matmul_dx(dy, w, off, dx_rows=m, dx=out)
        dx = out[at.cuda()]
        dw = bm.expert_matmul_dw(dy, x, off, x_rows=m)
        groups = [slice(0, 100), slice(100, 300)]
    else:
        # only the last rows are in groups
        first = rows - n + 5
        off = torch.tensor([first, first + 100, rows], dtype=torch.int32).cuda()
        full = torch.zeros(rows, N, dtype=BF, device="cuda")
        bm.expert_matmul(x, w, off, y=full)
        assert (full[:first] == 0).all()
        y = torch.cat([full[:5], full[first:]])
        fdy = torch.zeros(rows, N, dtype=BF, device="cuda")
        fdy[at.cuda()] = dy
        dx = bm.expert_matmul_dx(fdy, w, off, dx=torch.zeros(rows, K, dtype=BF, device="cuda"))[at.cuda()]
        dw = bm.expert_matmul_dw(fdy, x, off)
        groups = [slice(5, 105), slice(105, 300)]
    for e, s in enumerate(groups):
        d, wd = dy[s].double(), w[e].double()
        want, mag = xs[s] @ wd.t(), xs[s].abs() @ wd.abs().t()
        compare(y[s], want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(K) * mag, f"y {e}")
        want, mag = d @ wd, d.abs() @ wd.abs()
        compare(dx[s], want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(N) * mag, f"dx {e}")
        want, mag = d.t() @ xs[s], d.abs().t() @ xs[s].abs()
        compare(dw[e], want, ex.half_ulp(BF) * want.abs() + ex.sum_bound(200) * mag, f"dw {e}")


@pytest.mark.parametrize("T,N,K", [(2048, 1000, 4096), (300, 1001, 2056), (4096, 520, 264), (1024, 2048, 7168)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_large(bm, T, N, K, act):
    """Whole tiles and their edges with every part of the epilogue."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = large(g, T, K), large(g, N, K, scale=K ** -0.5)
    b, r = large(g, N), large(g, T, N)
    y, pre = bm.linear(x, w, bias=b, act=act, residual=r, keep_pre=True)
    z, mag = x.double() @ w.double().t() + b.double(), x.double().abs() @ w.double().abs().t() + b.double().abs()
    zb = ex.sum_bound(K + 1) * mag
    compare(pre, z, ex.half_ulp(BF) * z.abs() + zb, "pre")
    want = ex.act(z, act) + r.double()
    compare(y, want, ex.half_ulp(BF) * want.abs() + 1.13 * zb + 2.0 ** -18 * (z.abs() + 1) + 2.0 ** -23 * r.double().abs(),
            "y")


def test_offsets_are_kept_inside_the_call(bm):
    """Offsets outside [0, R] or descending cost wrong groups, never an access
    out of bounds (they are clamped): the buffers around stay as they were."""
    g = gen(9)
    x, _ = rnd(g, 40, 64)
    w, _ = rnd(g, 3, 128, 64)
    for off in ([-5, 10, 1000, 2 ** 31 - 1], [0, 30, 10, 40], [0, -7, -9, -1]):
        buf = torch.full((60, 128), 3.0, dtype=BF, device="cuda")
        bm.expert_matmul(x, w, torch.tensor(off, dtype=torch.int32).cuda(), y=buf[10:50])
        assert (buf[:10] == 3).all() and (buf[50:] == 3).all()
        dw = bm.expert_matmul_dw(buf[:40, :128], x, torch.tensor(off, dtype=torch.int32).cuda())
        assert dw.shape == (3, 128, 64)
    torch.cuda.synchronize()


def test_no_rows(bm):
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(2, 32, 64, dtype=BF, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert bm.expert_matmul(x, w, off).shape == (0, 32)
    dw = bm.expert_matmul_dw(torch.empty(0, 32, dtype=BF, device="cuda"), x, off,
                             dw=torch.full((2, 32, 64), 7.0, dtype=BF, device="cuda"))
    assert (dw == 0).all()
    y, _ = bm.linear(x, w[0])
    assert y.shape == (0, 32)
    dx, dw, db = bm.linear_backward(y, x, w[0], need_db=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    assert bm.swiglu(x, x).shape == (0, 64) and bm.combine(x, k=4).shape == (0, 64)


LINEAR = [(1, 256, 512, 0, 0), (1, 64, 7168, 0, 0), (5, 17, 33, 0, 0), (64, 128, 256, 0, 0), (130, 200, 72, 8, 8),
          (300, 96, 100, 3, 1), (257, 520, 1032, 0, 0), (16, 2048, 64, 0, 0), (33, 8, 4096, 0, 0)]


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("shape", LINEAR, ids=str)
def test_linear(bm, act, shape):
    T, N, K, pad, shift = shape
    dtype = HF if T % 2 else BF
    g = gen(T + N)
    x, x64 = rnd(g, T, K, dtype=dtype, pad=pad, shift=shift)
    w, w64 = rnd(g, N, K, dtype=dtype, scale=K ** -0.5, pad=pad, shift=shift)
    b = torch.randn(N, generator=g).to(dtype)
    r, r64 = rnd(g, T, N, dtype=dtype, pad=pad)
    say(f"[experts] linear {act} {shape} {dtype}")
    y, pre = bm.linear(x, w, bias=b.cuda(), act=act, residual=r, keep_pre=True)
    z, mag = x64 @ w64.t() + b.double(), x64.abs() @ w64.abs().t() + b.double().abs()
    zb = ex.sum_bound(K + 1) * mag
    check(pre, z, ex.half_ulp(dtype) * z.abs() + zb + 2.0 ** -24, f"linear {act} {shape} pre")
    want = ex.act(z, act) + r64
    # the activation: its slope is at most 1.13, its own evaluation within 2^-18 (|z| + 1)
    bound = ex.half_ulp(dtype) * want.abs() + 1.13 * zb + 2.0 ** -18 * (z.abs() + 1) + 2.0 ** -23 * r64.abs()
    check(y, want, bound, f"linear {act} {shape}")
    # onto a float32 residual in place, without bias
    s = torch.randn(T, N, generator=g)
    s64, sd = s.double(), s.cuda()
    y2, none = bm.linear(x, w, act=act, residual=sd, y=sd)
    assert y2 is sd and none is None
    z, mag = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    want = ex.act(z, act) + s64
    check(sd, want, 2.0 ** -24 * want.abs() + 1.13 * ex.sum_bound(K) * mag + 2.0 ** -18 * (z.abs() + 1) +
          2.0 ** -23 * s64.abs(), f"linear {act} {shape} in place")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("shape", LINEAR, ids=str)
def test_linear_backward(bm, act, shape):
    T, N, K, pad, shift = shape
    dtype = BF if T % 2 else HF
    g = gen(T + N + 7)
    x, x64 = rnd(g, T, K, dtype=dtype, pad=pad, shift=shift)
    w, w64 = rnd(g, N, K, dtype=dtype, scale=K ** -0.5, pad=pad, shift=shift)
    pre, p64 = rnd(g, T, N, dtype=dtype, scale=2.0, pad=pad)
    dy, dy64 = rnd(g, T, N, dtype=dtype, pad=pad)
    say(f"[experts] linear_backward {act} {shape} {dtype}")
    none = act == "none"
    dx, dw, db = bm.linear_backward(dy, x, w, act=act, pre=None if none else pre, need_db=True)
    dz = dy64 * ex.act_slope(p64, act)
    # dz: the slope within 2^-17, rounded once before the products
    ez = (0 if none else 2.0 ** -17) * dy64.abs()
    er = ez + (0 if none else ex.half_ulp(dtype)) * (dz.abs() + ez) + 2.0 ** -24 * (dtype == HF)
    m = dz.abs() + er
    u = ex.half_ulp(dtype)
    want = dz @ w64
    check(dx, want, u * (want.abs() + er @ w64.abs()) + er @ w64.abs() + ex.sum_bound(N) * (m @ w64.abs()) + 2.0 ** -24,
          f"linear_backward {act} {shape} dx")
    want = dz.t() @ x64
    check(dw, want, u * (want.abs() + er.t() @ x64.abs()) + er.t() @ x64.abs() + ex.sum_bound(T) * (m.t() @ x64.abs()) +
          2.0 ** -24, f"linear_backward {act} {shape} dw")
    want = dz.sum(0)
    check(db, want, u * (want.abs() + ez.sum(0)) + ez.sum(0) + ex.sum_bound(T) * m.sum(0) + 2.0 ** -24,
          f"linear_backward {act} {shape} db")
    # float32 gradients, one at a time, are those of a call for all
    a = bm.linear_backward(dy, x, w, act=act, pre=None if none else pre, out_dtype=F32, need_db=True)
    for i, want in enumerate(a):
        need = [j == i for j in range(3)]
        b = bm.linear_backward(dy, x, w, act=act, pre=None if none else pre, out_dtype=F32, need_dx=need[0],
                               need_dw=need[1], need_db=need[2])
        assert [t is not None for t in b] == need and torch.equal(b[i], want)


def test_slopes_of_far_values(bm):
    """Slopes where the exponentials and squares on their way overflow."""
    pre = torch.tensor([[-3e38, -1e20, -1e13, -200.0, 200.0, 1e13, 1e20, 3e38]], dtype=BF, device="cuda")
    one, x, w = torch.ones_like(pre), pre[:, :1], pre.new_zeros(8, 1)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        _, _, db = bm.linear_backward(one, x, w, act=act, pre=pre, need_dx=False, need_dw=False, need_db=True)
        assert db.tolist() == [0.0] * 4 + [1.0] * 4, act


@pytest.mark.parametrize("R,I,pad,shift", [(1, 1, 0, 0), (8, 2048, 0, 0), (3, 7, 0, 0), (300, 100, 4, 2), (70000, 8, 0, 0),
                                           (2, 4100, 0, 1)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_swiglu(bm, R, I, pad, shift, dtype):
    g = gen(R + I)
    z, z64 = rnd(g, R, 2 * I, dtype=dtype, scale=2.0, pad=pad, shift=shift)
    dh, d64 = rnd(g, R, I, dtype=dtype, pad=pad)
    gate, up, g64, u64 = z[:, :I], z[:, I:], z64[:, :I], z64[:, I:]
    say(f"[experts] swiglu R={R} I={I} {dtype}")
    u = ex.half_ulp(dtype)
    small = 2.0 ** -24 * (dtype == HF)          # half a step of fp16's smallest values
    want = ex.swiglu(g64, u64)
    h = bm.swiglu(gate, up)
    check(h, want, u * want.abs() + 2.0 ** -18 * want.abs() + small, "swiglu")
    dg, du = bm.swiglu_backward(dh, gate, up)
    wg, wu = ex.swiglu_backward(d64, g64, u64)
    check(dg, wg, u * wg.abs() + 2.0 ** -17 * (d64 * u64).abs() + small, "dgate")
    check(du, wu, u * wu.abs() + 2.0 ** -17 * wu.abs() + small, "dup")
    # in place: h over gate, then the gradients over their inputs
    gate2, up2 = gate.clone(), up.clone()
    assert bm.swiglu(gate2, up2, h=gate2) is gate2 and torch.equal(gate2, h)
    bm.swiglu_backward(dh, gate, up, dgate=gate, dup=up)
    assert torch.equal(gate, dg) and torch.equal(up, du)


def test_swiglu_far_values(bm):
    """Gates whose exponential overflows: silu is 0 or the gate itself."""
    gate = torch.tensor([[-3e38, -200.0, -88.8, 0.0, 88.8, 200.0, 3e38, -1e-30]], dtype=BF, device="cuda")
    one = torch.ones_like(gate)
    h = bm.swiglu(gate, one).cpu().double()
    assert torch.allclose(h, ex.act(gate.cpu().double(), "silu"), rtol=2 ** -8, atol=1e-30)
    dg, du = bm.swiglu_backward(one, gate, one)
    assert torch.isfinite(dg).all() and torch.isfinite(du).all()
    assert dg[0, :3].abs().max() < 1e-30 and (dg[0, 4:7] == 1).all() and dg[0, 3] == 0.5


@pytest.mark.parametrize("T,k,H,pad,shift", [(1, 8, 7168, 0, 0), (5, 1, 1, 0, 0), (33, 2, 100, 4, 0), (300, 16, 72, 0, 8),
                                             (70, 8, 513, 3, 1), (9, 3, 2050, 0, 0)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_combine(bm, T, k, H, pad, shift, dtype):
    g = gen(T + k + H)
    o, o64 = rnd(g, T * k, H, dtype=dtype, pad=pad, shift=shift)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    w64, wd = w.double(), w.cuda()
    r, r64 = rnd(g, T, H, dtype=dtype, pad=pad)
    u = ex.half_ulp(dtype)
    small = 2.0 ** -24 * (dtype == HF)
    say(f"[experts] combine T={T} k={k} H={H} {dtype}")
    want, mag = ex.combine(o64, w64, T, k, r64), ex.combine(o64.abs(), w64, T, k, r64.abs())
    check(bm.combine(o, wd, residual=r), want, u * want.abs() + ex.sum_bound(k + 1) * mag + small, "combine")
    want, mag = ex.combine(o64, torch.ones(T, k), T, k), ex.combine(o64.abs(), torch.ones(T, k), T, k)
    check(bm.combine(o, k=k), want, u * want.abs() + ex.sum_bound(k) * mag + small, "combine, no weights")
    s = torch.randn(T, H, generator=g)
    sd = s.cuda()
    want, mag = ex.combine(o64, w64, T, k, s.double()), ex.combine(o64.abs(), w64, T, k, s.double().abs())
    assert bm.combine(o, wd, residual=sd, y=sd) is sd
    check(sd, want, ex.sum_bound(k + 1) * mag, "combine in place, fp32")
    for dt in (dtype, F32):
        dy, dy64 = rnd(g, T, H, dtype=dt, pad=pad)
        do, dw = bm.combine_backward(dy, o, wd)
        wo, ww = ex.combine_backward(dy64, o64, w64, T, k)
        check(do, wo, u * wo.abs() + 2.0 ** -23 * wo.abs() + small, f"d_o, dy {dt}")
        _, mag = ex.combine_backward(dy64.abs(), o64.abs(), w64, T, k)
        check(dw, ww, ex.sum_bound(H) * mag, f"dw, dy {dt}")
        d1, none = bm.combine_backward(dy, o, wd, need_dw=False)
        assert none is None and torch.equal(d1, do)
        none, w1 = bm.combine_backward(dy, o, wd, need_do=False)
        assert none is None and torch.equal(w1, dw)
    # over o itself
    o2 = o.clone()
    d2, w2 = bm.combine_backward(dy, o2, wd, d_o=o2)
    assert torch.equal(o2, do) and torch.equal(w2, dw)


def test_combine_backward_of_the_most_tokens(bm):
    """2^24 tokens: more threads than one launch holds."""
    T, H = 2 ** 24, 520
    dy = torch.ones(T, H, dtype=BF, device="cuda")
    w = (torch.arange(T, device="cuda") % 251).float().view(T, 1)      # (below 256: exact in bfloat16)
    do, dw = bm.combine_backward(dy, dy, w)
    assert (dw == H).all()
    for t in range(0, T, 2 ** 22):
        assert (do[t:t + 2 ** 22] == w[t:t + 2 ** 22].to(BF)).all()


def layer(bm, x, wgu, wd, ids, wt, res, E, k):
    """The expert layer forward, as a user chains it."""
    I = wd.shape[2]
    _, off, perm, _, _ = bm.bucket(ids, E)
    z = bm.expert_matmul(x, wgu, off, x_rows=perm, x_div=k)
    h = bm.swiglu(z[:, :I], z[:, I:])
    o = bm.expert_matmul(h, wd, off, y_rows=perm)
    return off, perm, z, h, o, bm.combine(o, wt, residual=res)


def layer_backward(bm, dy, x, wgu, wd, wt, off, perm, z, h, o, k):
    I = wd.shape[2]
    do, dwt = bm.combine_backward(dy, o, wt)
    dh = bm.expert_matmul_dx(do, wd, off, dy_rows=perm)
    dwd = bm.expert_matmul_dw(do, h, off, dy_rows=perm)
    dg, du = bm.swiglu_backward(dh, z[:, :I], z[:, I:])
    dz = dg.as_strided((dg.shape[0], 2 * I), (2 * I, 1))
    dxp = bm.expert_matmul_dx(dz, wgu, off, dx_rows=perm)
    dwgu = bm.expert_matmul_dw(dz, x, off, x_rows=perm, x_div=k)
    return bm.combine(dxp, k=k), dwgu, dwd, dwt


def run_layer(bm, x, wgu, wd, ids, wt, res, dy, E, k):
    off, perm, z, h, o, y = layer(bm, x, wgu, wd, ids, wt, res, E, k)
    return (y,) + layer_backward(bm, dy, x, wgu, wd, wt, off, perm, z, h, o, k)


def layer_inputs(T, H, I, E, k, dtype, seed=3):
    g = gen(seed)
    t = {"x": rnd(g, T, H, dtype=dtype), "wgu": rnd(g, E, 2 * I, H, dtype=dtype, scale=H ** -0.5),
         "wd": rnd(g, E, H, I, dtype=dtype, scale=I ** -0.5), "res": rnd(g, T, H, dtype=dtype),
         "dy": rnd(g, T, H, dtype=dtype)}
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    wt = torch.softmax(torch.randn(T, k, generator=g), 1)
    return t, ids, wt


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 512, 8, 2), (33, 256, 128, 8, 2), (150, 264, 96, 5, 3)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_expert_layer_forward_and_backward(bm, T, H, I, E, k, dtype):
    """The operators together, against autograd of the layer in float64.  In
    the norm of each output: a chain of at most 8 roundings to the type (z, h,
    o, y; do, dh, dz, dx and what they multiply), each carried on with a gain
    of at most 2 (slopes of SwiGLU below 1.13, products of both factors)."""
    t, ids, wt = layer_inputs(T, H, I, E, k, dtype)
    got = run_layer(bm, *(t[n][0] for n in ("x", "wgu", "wd")), ids.cuda(), wt.cuda(), t["res"][0], t["dy"][0], E, k)
    x, wgu, wd, w64 = (v.clone().requires_grad_() for v in (t["x"][1], t["wgu"][1], t["wd"][1], wt.double()))
    y = t["res"][1].clone()
    for j in range(k):
        e = ids[:, j].long()
        z = (wgu[e] @ x[:, :, None])[:, :, 0]
        y = y + w64[:, j:j + 1] * (wd[e] @ ex.swiglu(z[:, :I], z[:, I:])[:, :, None])[:, :, 0]
    (y * t["dy"][1]).sum().backward()
    for name, a, b in zip(("y", "dx", "dwgu", "dwd", "dweights"), got,
                          (y.detach(), x.grad, wgu.grad, wd.grad, w64.grad)):
        rel = ((a.cpu().double() - b).norm() / b.norm()).item()
        say(f"[experts] layer T={T} {dtype} {name}: relative error {rel:.2e}")
        assert rel <= 16 * ex.half_ulp(dtype), name


def test_layer_captured_and_replayed(bm):
    """The layer captured into a graph, replayed with eager work and new
    inputs between the replays; two graphs at once."""
    E, k, T, H, I = 8, 2, 40, 256, 128
    t, ids, wt = layer_inputs(T, H, I, E, k, BF)
    args = [t["x"][0], t["wgu"][0], t["wd"][0], ids.cuda(), wt.cuda(), t["res"][0], t["dy"][0]]
    run_layer(bm, *args, E, k)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run_layer(bm, *args, E, k)
        graphs.append((g, out))
    for i in range(4):
        t2, ids2, wt2 = layer_inputs(T, H, I, E, k, BF, seed=20 + i)
        for dst, src in zip(args, [t2["x"][0], t2["wgu"][0], t2["wd"][0], ids2.cuda(), wt2.cuda(), t2["res"][0],
                                   t2["dy"][0]]):
            dst.copy_(src)
        for g, _ in graphs:
            g.replay()
        want = run_layer(bm, *args, E, k)
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_other_streams(bm):
    """Calls on given streams, at once, give what the current stream gives."""
    g = gen(4)
    x, _ = rnd(g, 200, 512)
    w, _ = rnd(g, 4, 256, 512)
    off = offsets_of([60, 0, 100, 40]).cuda()
    want = bm.expert_matmul(x, w, off)
    lin, _ = bm.linear(x, w[1], act="gelu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [(bm.expert_matmul(x, w, off, stream=s), bm.linear(x, w[1], act="gelu", stream=s)[0]) for s in streams]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, lin)


def test_binding_refusals(bm):
    c = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    i32 = lambda n: c(n, dt=torch.int32)  # noqa: E731
    x, w, off = c(4, 8), c(2, 16, 8), i32(3)
    for f in (lambda: bm.expert_matmul(c(4, 9), w, off), lambda: bm.expert_matmul(x, w, i32(4)),
              lambda: bm.expert_matmul(x, w, off, x_rows=i32(3), y_rows=i32(4)),
              lambda: bm.expert_matmul(x, w, off, y_rows=i32(5)),
              lambda: bm.expert_matmul(x, w, off, x_rows=i32(8)[::2]),
              lambda: bm.expert_matmul(c(8, 4).t(), w, off), lambda: bm.expert_matmul(x[:1].expand(4, 8), w, off),
              lambda: bm.expert_matmul(x, w, off, y=c(4, 16), out_dtype=F32),
              lambda: bm.expert_matmul_dw(c(5, 16), x, off), lambda: bm.expert_matmul_dw(c(4, 16), x, off, accumulate=True),
              lambda: bm.expert_matmul_dw(c(4, 16), x, off, dw=c(2, 8, 16)), lambda: bm.linear(x, w[0], bias=c(15)),
              lambda: bm.linear(x, w[0], residual=c(4, 15)), lambda: bm.linear_backward(c(4, 16), x, w[0], act="silu"),
              lambda: bm.linear_backward(c(4, 16), c(5, 8), w[0]), lambda: bm.swiglu(x, c(4, 9)),
              lambda: bm.swiglu_backward(x, x, x, dgate=x), lambda: bm.combine(x), lambda: bm.combine(x, k=3),
              lambda: bm.combine(x, c(2, 2)), lambda: bm.combine_backward(c(2, 8), None, c(2, 2, dt=F32)),
              lambda: bm.combine(x, k=2, residual=c(3, 8))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        bm.expert_matmul(c(4, 8, dt=torch.float32), w, off)
    with pytest.raises(bm.BitMoEError):
        bm.expert_matmul(x, w, off, y=c(3, 16))
    with pytest.raises(bm.BitMoEError):
        bm.expert_matmul(x, w, off, x_rows=i32(4), x_div=0)
    torch.cuda.synchronize()
