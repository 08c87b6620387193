"""A share of the experts, as each process of an expert-parallel layer runs it:
bucket's offsets from the share's first expert on, its whole perm."""
import pytest

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


def leave_nan(*shape, dtype):
    """Memory that the next allocation of this size finds full of NaN."""
    for _ in range(2):
        torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def inputs(T, k, E, N, K, dtype):
    g = torch.Generator().manual_seed(T + E)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    make = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    return ids, make


@pytest.mark.parametrize("T,k,E,N,K", [(1, 2, 8, 128, 64), (40, 4, 16, 200, 264), (300, 3, 6, 65, 39), (2000, 8, 64, 512, 256)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_rows_of_other_shares_are_zero(bm, T, k, E, N, K, dtype):
    ids, make = inputs(T, k, E, N, K, dtype)
    x, w, dy = make(T, K), make(E, N, K), make(T * k, N)
    _, off, perm, _, _ = bm.bucket(ids, E)
    y = bm.expert_matmul(x, w, off, x_rows=perm, x_div=k, y_rows=perm)
    dx = bm.expert_matmul_dx(dy, w, off, dy_rows=perm, dx_rows=perm)
    pair = ids.flatten().long()
    say(f"[experts] shares T={T} k={k} E={E} N={N} K={K} {dtype}")
    for e0, e1 in ((0, E // 2), (E // 2, E), (1, 2), (0, E)):
        mine = ((pair >= e0) & (pair < e1))[:, None]
        for out in (dtype, F32):
            leave_nan(T * k, N, dtype=out)
            got = bm.expert_matmul(x, w[e0:e1], off[e0:e1 + 1], x_rows=perm, x_div=k, y_rows=perm, out_dtype=out)
            assert ((got == 0) | mine).all()
            if out == dtype:
                # (a share may take another kernel: the sums' order is not the whole layer's)
                assert torch.allclose(got.float(), torch.where(mine, y, 0).float(), rtol=2 ** -6, atol=2 ** -6 * K ** 0.5)
            leave_nan(T * k, K, dtype=out)
            got = bm.expert_matmul_dx(dy, w[e0:e1], off[e0:e1 + 1], dy_rows=perm, dx_rows=perm, out_dtype=out)
            assert ((got == 0) | mine).all()
            if out == dtype:
                assert torch.allclose(got.float(), torch.where(mine, dx, 0).float(), rtol=2 ** -6, atol=2 ** -6 * N ** 0.5)


def test_shares_combined_are_the_layer(bm):
    """The sum over the shares of each one's combine, as an all-reduce gives
    it."""
    T, k, E, N, K = 100, 4, 12, 96, 128
    ids, make = inputs(T, k, E, N, K, BF)
    x, w = make(T, K), make(E, N, K)
    wt = torch.rand(T, k, device="cuda")
    _, off, perm, _, _ = bm.bucket(ids, E)
    total = torch.zeros(T, N, device="cuda")
    for e0, e1 in ((0, 5), (5, 6), (6, 12)):
        leave_nan(T * k, N, dtype=BF)
        o = bm.expert_matmul(x, w[e0:e1], off[e0:e1 + 1], x_rows=perm, x_div=k, y_rows=perm)
        total += bm.combine(o, wt, out_dtype=F32)
    rows = (w[ids.flatten().long()].float() @ x.repeat_interleave(k, 0).float()[:, :, None])[:, :, 0]
    want = (rows.view(T, k, N) * wt[:, :, None]).sum(1)
    # each pair's row rounded once to bfloat16, the combine's and the sums' own roundings far below
    bound = (rows.abs().view(T, k, N) * wt[:, :, None]).sum(1) * 2.0 ** -8 * 1.01 + 2.0 ** -10
    assert ((total - want).abs() <= bound).all()


def test_given_output_keeps_what_it_held(bm):
    """A y that the caller gives is written where a group's row goes, nowhere
    else, as without a share; clear_ungrouped's own borders, strides and maps."""
    T, k, E, N, K = 50, 2, 6, 40, 64
    ids, make = inputs(T, k, E, N, K, BF)
    x, w = make(T, K), make(E, N, K)
    _, off, perm, _, _ = bm.bucket(ids, E)
    y = torch.full((T * k, N), 7.0, dtype=BF, device="cuda")
    bm.expert_matmul(x, w[2:4], off[2:5], x_rows=perm, x_div=k, y_rows=perm, y=y)
    pair = ids.flatten().long()
    assert (y[(pair < 2) | (pair >= 4)] == 7).all()
    # a map that takes some rows away: the row that they would have had stays undefined, no access is out of bounds
    gone = perm.clone()
    gone[::3] = -1
    gone[1::7] = T * k + 5
    leave_nan(T * k, N, dtype=BF)
    got = bm.expert_matmul(x, w[2:4], off[2:5], x_rows=perm, x_div=k, y_rows=gone)
    lo, hi = int(off[2]), int(off[4])
    for r in list(range(lo)) + list(range(hi, T * k)):
        if 0 <= int(gone[r]) < T * k:
            assert (got[int(gone[r])] == 0).all()
    torch.cuda.synchronize()


def test_share_captured_and_replayed(bm):
    T, k, E, N, K = 64, 4, 8, 128, 256
    ids, make = inputs(T, k, E, N, K, BF)
    x, w, wt = make(T, K), make(E, N, K), torch.rand(T, k, device="cuda")

    def run():
        _, off, perm, _, _ = bm.bucket(ids, E)
        o = bm.expert_matmul(x, w[2:5], off[2:6], x_rows=perm, x_div=k, y_rows=perm)
        return o, bm.combine(o, wt)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for i in range(4):
        ids.copy_(torch.stack([torch.randperm(E)[:k] for _ in range(T)]).to(torch.int32))
        x.normal_()
        out[0].fill_(float("nan"))
        g.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
