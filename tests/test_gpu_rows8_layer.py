"""The operators in 8 bits and the block norms together, as they are used around
the expert layer: served in 8 bits, and a training step that keeps its activations
in 8 bits; captured, on other streams, several calls at once."""
import pytest

import _experts as ex
import _rows8 as r8
from _gpu import require_gpu, say, torch
from test_gpu_experts import BF, F32, HF, gen, rnd

pytestmark = pytest.mark.gpu
EPS, SCALE = 1e-6, 0.875


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def inputs(T, H, I, E, k, dtype, seed=3):
    g = gen(seed)
    one = lambda: (lambda v: (v.cuda(), v.double()))((1 + 0.1 * torch.randn(H, generator=g)).to(dtype))  # noqa: E731
    t = {"x": rnd(g, T, H, dtype=dtype), "wgu": rnd(g, E, 2 * I, H, dtype=dtype, scale=H ** -0.5),
         "wd": rnd(g, E, H, I, dtype=dtype, scale=I ** -0.5), "before": one(), "after": one(), "next": one(), "gate": one(),
         "ds": rnd(g, T, H, dtype=dtype), "dn": rnd(g, T, H, dtype=dtype)}
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    t["wt"] = (lambda v: (v.cuda(), v.double()))(torch.softmax(torch.randn(T, k, generator=g), 1))
    return t, ids


def serve(bm, t, wgu, wd, ids, E, k):
    """norm, experts in 8 bits, combine, norm, gate and stream: (combine's rows,
    the stream, the next block's input)."""
    d = {n: v[0] for n, v in t.items()}
    I = wd.codes.shape[2]
    _, n = bm.block_norm(None, d["x"], w_before=d["before"], eps=EPS, need_s=False)
    _, off, perm, _, _ = bm.bucket(ids, E)
    z = bm.expert_matmul_i8(bm.quantize_rows(n), wgu, off, x_rows=perm, x_div=k, out_dtype=n.dtype)
    h = bm.swiglu_rows8(z[:, :I], z[:, I:])
    y = bm.combine(bm.expert_matmul_i8(h, wd, off, y_rows=perm, out_dtype=n.dtype), d["wt"])
    return (y,) + tuple(bm.block_norm(y, d["x"], w_after=d["after"], gate=d["gate"], scale=SCALE, w_before=d["next"], eps=EPS))


def step(bm, t, ids, E, k, block=32):
    """A training step around 16-bit experts: the activation's inputs kept in 8
    bits, the down projection's weights' gradient from what they stand for."""
    d = {n: v[0] for n, v in t.items()}
    I = d["wd"].shape[2]
    _, n = bm.block_norm(None, d["x"], w_before=d["before"], eps=EPS, need_s=False)
    _, off, perm, _, _ = bm.bucket(ids, E)
    z = bm.expert_matmul(n, d["wgu"], off, x_rows=perm, x_div=k)
    h, g8, u8 = bm.swiglu_checkpoint(z[:, :I], z[:, I:], block=block)
    o = bm.expert_matmul(h, d["wd"], off, y_rows=perm)
    y = bm.combine(o, d["wt"])
    s, m = bm.block_norm(y, d["x"], w_after=d["after"], gate=d["gate"], scale=SCALE, w_before=d["next"], eps=EPS)
    b = bm.block_norm_backward(d["dn"], d["ds"], s, y, w_after=d["after"], gate=d["gate"], scale=SCALE, w_before=d["next"], eps=EPS)
    do, dwt = bm.combine_backward(b.d_o, o, d["wt"])
    dh = bm.expert_matmul_dx(do, d["wd"], off, dy_rows=perm)
    dg, du, h = bm.swiglu_checkpoint_backward(dh, g8, u8, need_h=True)
    dwd = bm.expert_matmul_dw(do, h, off, dy_rows=perm)
    dz = dg.as_strided((dg.shape[0], 2 * I), (2 * I, 1))
    dn = bm.combine(bm.expert_matmul_dx(dz, d["wgu"], off, dx_rows=perm), k=k)
    dwgu = bm.expert_matmul_dw(dz, n, off, x_rows=perm, x_div=k)
    a = bm.block_norm_backward(dn, b.dresidual, d["x"], w_before=d["before"], eps=EPS)
    return {"s": s, "n": m, "x": a.dresidual, "before": a.dw_before, "wgu": dwgu, "wd": dwd, "wt": dwt, "after": b.dw_after,
            "gate": b.dgate, "next": b.dw_before}


def chain(v, ids, k):
    """The block in float64: (the experts' input, gate and up of every pair, their h,
    the pairs' outputs [k, T, H], combine's rows, the stream, the next block's input)."""
    n = r8.block_norm(None, v["x"], None, None, 1.0, v["before"], EPS)[1]
    I = v["wd"].shape[2]
    zs, hs, os, y = [], [], [], 0
    for j in range(k):
        e = ids[:, j].long()
        z = (v["wgu"][e] @ n[:, :, None])[:, :, 0]
        h = ex.swiglu(z[:, :I], z[:, I:])
        zs.append(z)
        hs.append(h)
        os.append((v["wd"][e] @ h[:, :, None])[:, :, 0])
        y = y + v["wt"][:, j:j + 1] * os[-1]
    return (n, torch.cat(zs), torch.cat(hs), torch.stack(os), y) + r8.block_norm(y, v["x"], v["after"], v["gate"], SCALE, v["next"], EPS)


def code_error(v, block=0):
    """Half a code's step over all values against the values, in the norm."""
    b = r8.blocks_of(v, block)
    half = (b.abs().amax(2) / 254).square().sum() * b.shape[2]
    return float((half / v.square().sum()).sqrt())


SIZES = [(1, 256, 512, 8, 2), (33, 256, 128, 8, 2), (150, 264, 96, 5, 3), (40, 250, 75, 6, 2)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_block_served_in_8_bits(bm, T, H, I, E, k, dtype):
    """Against the block in float64 with the weights that the codes stand for.  In
    the norm of each output: at most 8 roundings to the type with gains of at most 2,
    as for the 16-bit layer; n's codes off by half a step each, which gate and up
    carry on, both times (2, and 1.13 for silu's slope); h's codes the same once.  The
    last norm's length may add its own share (2)."""
    t, ids = inputs(T, H, I, E, k, dtype)
    wgu, wd = bm.quantize_rows(t["wgu"][0]), bm.quantize_rows(t["wd"][0])
    got = serve(bm, t, wgu, wd, ids.cuda(), E, k)
    v = {n: x[1] for n, x in t.items()}
    for name, w in (("wgu", wgu), ("wd", wd)):
        v[name] = w.codes.cpu().double() * w.scale.cpu().double()[:, :, None]
    n, z, h, _, *want = chain(v, ids, k)
    bound = 2 * (16 * ex.half_ulp(dtype) + 2.3 * code_error(n) + code_error(h))
    for name, a, b in zip(("combine", "stream", "next"), got, want):
        rel = ((a.cpu().double() - b).norm() / b.norm()).item()
        say(f"[rows8] served T={T} {dtype} {name}: relative error {rel:.2e} of {bound:.2e}")
        assert rel <= bound, name


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_training_step_with_kept_activations(bm, T, H, I, E, k, dtype):
    """Against autograd of the block in float64.  In the norm of each output: 16
    roundings' worth as for the 16-bit layer, and twice that for the norms' own (their
    projections may cancel half of a gradient); what is kept is off by half a code's
    step, which the backward's products of slopes and factors carry on with a gain of
    at most 4.  The combine weights' gradients are products of two rows that may be
    nearly orthogonal (the norm's projection makes them so: sum_j w_j <dy, o_j> is
    about 0), so their errors are against the rows' lengths: |<dy + e, o + f> - <dy, o>|
    <= |e| |o| + |dy| |f| + |e| |f|."""
    t, ids = inputs(T, H, I, E, k, dtype)
    got = step(bm, t, ids.cuda(), E, k)
    leaves = {n: x[1].clone().requires_grad_(n not in ("ds", "dn")) for n, x in t.items()}
    n, z, h, o, y, s, m = chain(leaves, ids, k)
    y.retain_grad()
    ((s * leaves["ds"]).sum() + (m * leaves["dn"]).sum()).backward()
    bound = 32 * ex.half_ulp(dtype) + 4 * code_error(z.detach(), 32)
    for name, a in got.items():
        b = (s if name == "s" else m).detach() if name in ("s", "n") else leaves[name].grad
        length = b.norm() if name != "wt" else (y.grad.norm(dim=1) * o.detach().norm(dim=2)).norm()
        rel = ((a.cpu().double() - b).norm() / length).item()
        say(f"[rows8] step T={T} {dtype} {name}: relative error {rel:.2e} of {bound:.2e}")
        assert rel <= bound, name


def test_captured_and_replayed(bm):
    """Both captured into graphs, two of each (with workspaces of their own),
    replayed with eager work and new inputs between the replays."""
    E, k, T, H, I = 8, 2, 40, 256, 130
    t, ids = inputs(T, H, I, E, k, BF)
    ids = ids.cuda()
    wgu, wd = bm.quantize_rows(t["wgu"][0]), bm.quantize_rows(t["wd"][0])

    def run():
        return list(serve(bm, t, wgu, wd, ids, E, k)) + list(step(bm, t, ids, E, k).values())
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for i in range(4):
        t2, ids2 = inputs(T, H, I, E, k, BF, seed=30 + i)
        for name in t:
            t[name][0].copy_(t2[name][0])
        ids.copy_(ids2)
        bm.quantize_rows(t["wgu"][0].view(-1, H), out=bm.Rows8(wgu.codes.view(-1, H), wgu.scale.view(-1)))
        for g, _ in graphs:
            g.replay()
        want = run()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_other_streams_and_calls_at_once(bm):
    """Calls on given streams, at once, give what the current stream gives."""
    g = gen(4)
    x, _ = rnd(g, 200, 512)
    w = bm.quantize_rows(rnd(g, 4, 264, 512)[0])
    odd = bm.quantize_rows(rnd(g, 4, 33, 511)[0])
    off = torch.tensor([0, 60, 60, 160, 200], dtype=torch.int32, device="cuda")
    wt = torch.ones(512, dtype=BF, device="cuda")

    def run(s=None):
        q, r = bm.quantize_rows(x, stream=s), bm.quantize_rows(x[:, :511], stream=s)
        h, g8, u8 = bm.swiglu_checkpoint(x[:, :256], x[:, 256:], stream=s)
        b = bm.block_norm_backward(x, x, x, x, w_after=wt, gate=wt, w_before=wt, stream=s)
        return [bm.expert_matmul_i8(q, w, off, stream=s), bm.expert_matmul_i8(r, odd, off, stream=s),
                bm.expert_matmul_i8(bm.Rows8(q.codes[:3], q.scale[:3]), bm.Rows8(w.codes[0], w.scale[0]), stream=s),
                bm.dequantize_rows(q, stream=s), *bm.swiglu_rows8(x[:, :256], x[:, 256:], stream=s)[:2], h,
                *bm.swiglu_checkpoint_backward(x[:, :256], g8, u8, stream=s)[:2],
                *bm.block_norm(x, x, w_after=wt, gate=wt, w_before=wt, stream=s), *b]
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [run(s) for s in streams]
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_binding_refusals(bm):
    c = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    x = c(8, 64)
    q = bm.quantize_rows(x)
    w = bm.quantize_rows(c(2, 16, 64))
    off = c(3, dt=torch.int32)
    for f in (lambda: bm.expert_matmul_i8(q, w, off, y=c(7, 16)), lambda: bm.expert_matmul_i8(q, w, off, x_rows=c(8, dt=torch.int32), x_div=0),
              lambda: bm.expert_matmul_i8(q, w, off, ws=c(0, dt=torch.uint8), y=c(8, 16), x_rows=c(8, dt=torch.int32), x_div=0),
              lambda: bm.block_norm(x, eps=0.0), lambda: bm.block_norm_backward(x, x, x, x, eps=-1.0),
              lambda: bm.block_norm(c(1, 16385)), lambda: bm.block_norm_backward(x, x, w_before=c(64))):
        with pytest.raises(bm.BitMoEError):
            f()
    with pytest.raises(ValueError):
        bm.expert_matmul_i8(bm.Rows8(q.codes, q.scale.cpu()), w, off)
    torch.cuda.synchronize()
