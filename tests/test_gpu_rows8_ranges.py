"""The operators in 8 bits and the norms at sizes that take other instances of their
kernels or other paths in them than small ones do: loads and stores past the memory-side
cache, more rows than one launch holds, several rows a workgroup, every pair of tile and
parts.  Against float64, on the device; bounds: _rows8.py."""
import pytest

import _experts as ex
import _rows8 as r8
import _rows8_pairs as pairs
from _gpu import require_gpu, say, torch
from test_gpu_experts import BF, F32, HF
from test_gpu_rows8_kernels import ident
from test_gpu_rows8_kernels import test_every_kernel as compare_product

pytestmark = pytest.mark.gpu
MIB = 1 << 20
EPS = 1e-6


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, R, C, dtype, pad=0, scale=1.0):
    """[R, C] on the device, rows C + pad apart, the first one element behind an aligned
    address where there is a pad."""
    shift = 1 if pad else 0
    buf = torch.full((R * (C + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    t = buf[shift:].as_strided((R, C), (C + pad, 1))
    for r in range(0, R, 1 << 16):
        v = t[r:r + (1 << 16)]
        v.copy_(torch.randn(v.shape, generator=g, device="cuda") * scale)
    return t


def near(got, want, bound, what):
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    err = (got.double() - want).abs()
    worst = (err / (bound + 1e-300)).max().item()
    say(f"[ranges] {what}: largest error {worst:.2f} of its bound")
    assert worst <= 1, what


def chunks(R):
    return [slice(r, min(r + (1 << 14), R)) for r in range(0, R, 1 << 14)]


@pytest.mark.parametrize("case", pairs.I8, ids=ident)
def test_products(bm, case):
    compare_product(bm, case)


# rows at which 3 bytes an element are past 288 and 768 MiB
@pytest.mark.parametrize("R", [49300, 131200])
@pytest.mark.parametrize("dtype,C,pad", [(BF, 2047, 2), (HF, 2048, 0), (F32, 2047, 2)], ids=["bf16", "fp16", "fp32"])
def test_rows(bm, R, dtype, C, pad):
    assert 3 * R * C >= (288 if R < 1e5 else 768) * MIB
    x = rnd(gen(R), R, C, dtype, pad)
    y = {t: rnd(gen(1), R, C, t, pad) for t in (BF, HF, F32)}
    for block in (0, 32, 64, 128):
        say(f"[ranges] rows {R} x {C} {dtype} block {block}")
        q = bm.quantize_rows(x, block=block)
        for s in chunks(R):
            t, codes, scale = r8.quantize(x[s].double(), block)
            if dtype is F32:
                assert ((q.codes[s].double() - t).abs() <= 0.5 + 127 * 2 * r8.U).all()
            else:
                assert torch.equal(q.codes[s], codes.to(torch.int8))
            got = q.scale[s] if block else q.scale[s][:, None]
            assert ((got.double() - scale).abs() <= r8.U * scale).all()
        wide = q.scale.repeat_interleave(block, 1)[:, :C] if block else q.scale[:, None]
        for to, v in y.items():
            bm.dequantize_rows(q, y=v)
            assert all(torch.equal(v[s], (q.codes[s].float() * wide[s]).to(to)) for s in chunks(R)), to


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_swiglu_rows8(bm, dtype):
    R, I = 49300, 2047
    z = rnd(gen(2), R, 2 * I, dtype, scale=2.0)
    for block in (0, 64):
        q = bm.swiglu_rows8(z[:, :I], z[:, I:], block=block)
        for s in chunks(R):
            g, u = z[s, :I].double(), z[s, I:].double()
            h = ex.swiglu(g, u)
            e = (r8.silu_bound(g) + r8.U) * h.abs()
            scale = r8.quantize(h, block)[2]
            got = q.scale[s] if block else q.scale[s][:, None]
            near(got, scale, r8.blocks_of(e, block).amax(2) / 127 + r8.U * scale, "scales")
            wide = got.double().repeat_interleave(block or I, 1)[:, :I]
            near(q.codes[s].double() * wide, h, wide * (0.5 + 127 * 3 * r8.U) + e, "values")


# 8 bytes an element are past 288 and 768 MiB
@pytest.mark.parametrize("R,I", [(18600, 2047), (49200, 2048)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_checkpoint(bm, R, I, dtype):
    assert 8 * R * I >= (288 if R < 2e4 else 768) * MIB
    z, dh = rnd(gen(3), R, 2 * I, dtype, scale=2.0), rnd(gen(4), R, I, dtype, 2)
    gate, up = z[:, :I], z[:, I:]
    u = ex.half_ulp(dtype) * (1 + 2.0 ** -8)
    small = 2.0 ** -25 * (dtype is HF)
    for block in (32, 64, 128):
        say(f"[ranges] checkpoint {R} x {I} {dtype} block {block}")
        h, g8, u8 = bm.swiglu_checkpoint(gate, up, block=block)
        for got, x in ((g8, gate), (u8, up)):
            q = bm.quantize_rows(x, block=block)
            assert torch.equal(got.codes, q.codes) and torch.equal(got.scale, q.scale)
        dg, du, h8 = bm.swiglu_checkpoint_backward(dh, g8, u8, need_h=True)
        for s in chunks(R):
            g = gate[s].double()
            want = ex.swiglu(g, up[s].double())
            near(h[s], want, (u + r8.silu_bound(g) + r8.U) * want.abs() + small, "h")
            gk, uk = (r8.values(q.codes[s].double(), q.scale[s].double(), block) for q in (g8, u8))
            d = dh[s].double()
            wg, wu = ex.swiglu_backward(d, gk, uk)
            wh = ex.swiglu(gk, uk)
            near(dg[s], wg, u * wg.abs() + r8.slope_bound(d, gk, uk) + small, "dgate")
            near(du[s], wu, (u + r8.silu_bound(gk) + 3 * r8.U) * wu.abs() + small, "dup")
            near(h8[s], wh, (u + r8.silu_bound(gk) + 3 * r8.U) * wh.abs() + small, "h again")


def test_more_rows_than_a_launch(bm):
    """2^21 rows are one launch of the quantiser by rows and of the norm."""
    R, C = (1 << 21) + 3, 24
    x = rnd(gen(5), R, C, BF)
    q = bm.quantize_rows(x)
    t, codes, scale = r8.quantize(x.double())
    assert torch.equal(q.codes, codes.to(torch.int8))
    near(q.scale[:, None], scale, r8.U * scale, "scales")
    w, one = torch.randn(C, generator=gen(6), device="cuda").to(BF), torch.ones(1, dtype=r8.F64, device="cuda")
    s, n = bm.block_norm(x, x, w_after=w, scale=0.875, eps=EPS)
    ws, wn, es, en = r8.norm_bounds(x.double(), x.double(), w.double(), one, 0.875, one, EPS, BF, BF)
    near(s, ws, es, "s")
    near(n, wn, en, "n")


def norm_backward(bm, T, H, pad, dtype, stream, gate, huge=()):
    """block_norm_backward against float64; huge: rows of s and o whose squares leave
    float32."""
    g = gen(T + H)
    d = {"dn": rnd(g, T, H, dtype, pad), "ds": rnd(g, T, H, stream, pad), "s": rnd(g, T, H, stream, pad, 2.0), "o": rnd(g, T, H, dtype, pad)}
    for r in set(huge):
        d["s"][r] *= 1e25
        d["o"][r] *= 1e25
    wa, wb, gc = (torch.randn(H, generator=g, device="cuda").to(dtype) for _ in range(3))
    gt = gc if gate == "channel" else rnd(g, T, H, dtype, pad)
    say(f"[ranges] norm backward {T} x {H} {dtype} {stream} gate by {gate}")
    got = bm.block_norm_backward(d["dn"], d["ds"], d["s"], d["o"], w_after=wa, gate=gt, scale=0.875, w_before=wb, eps=EPS, out_dtype=F32)
    want, bound = r8.norm_backward_bounds(*(d[k].double() for k in ("dn", "ds", "s", "o")), wa.double(), gt.double(), 0.875,
                                          wb.double(), EPS, dtype, stream, F32)
    for name in ("d_o", "dresidual", "dw_after", "dw_before", "dgate"):
        at = "dgate_sum" if name == "dgate" and gate == "channel" else name
        # (a huge row's gradients of o are near float32's smallest normal values)
        near(getattr(got, name), want[at], bound[at] + (1e-36 if huge else 0), name)


TYPES = pytest.mark.parametrize("dtype,stream", [(BF, BF), (HF, HF), (BF, F32), (HF, F32)], ids=["bf16", "fp16", "bf16-fp32", "fp16-fp32"])
GATES = pytest.mark.parametrize("gate", ["channel", "token"])


@pytest.mark.parametrize("T,H,pad", [(13000, 2047, 2), (3600, 7168, 0)])
@TYPES
@GATES
def test_norm_backward_past_the_cache(bm, T, H, pad, dtype, stream, gate):
    assert 12 * T * H >= 288 * MIB
    norm_backward(bm, T, H, pad, dtype, stream, gate)


# (rows of a workgroup at a time, workgroups): two steps and a part of a third
@pytest.mark.parametrize("T,H,groups,most", [(7001, 300, 4, 768), (3501, 1000, 2, 768), (1601, 2047, 1, 768), (1100, 4000, 1, 512),
                                             (561, 7168, 1, 256), (515, 8200, 1, 256)])
@TYPES
@GATES
def test_norm_backward_rows_in_turn(bm, T, H, groups, most, dtype, stream, gate):
    """Workgroups that take several rows one after another, in bfloat16 with rows whose
    squares leave float32 first, last, one behind another and beside others."""
    step = groups * most
    huge = [0, step, groups + step + 1, 2 * groups, 2 * groups + 2 * step, 3 * groups + groups - 1, T - 1] if dtype is BF else []
    assert all(r < T for r in huge) and 2 * step < T <= 3 * step
    norm_backward(bm, T, H, 0, dtype, stream, gate, huge)


def test_gates_far_below_zero(bm):
    """silu(z) down to float32's smallest normal value (z = -92), and past it: e^z is
    itself below that from z = -87.3.  Behind its relative error a value has float32's and
    bfloat16's steps near 0 (2^-149 times what it is taken times; half of 2^-133)."""
    z = -torch.arange(80, 106, 0.5)
    gate = z[:, None].repeat(1, 96).to(BF).cuda()
    up, dh = rnd(gen(7), z.numel(), 96, BF), rnd(gen(8), z.numel(), 96, BF)
    g, u, d = gate.double(), up.double(), dh.double()
    half, zero = ex.half_ulp(BF) * (1 + 2.0 ** -8), 2.0 ** -134
    say("[ranges] gates from -80 to -105.5")
    h, g8, u8 = bm.swiglu_checkpoint(gate, up, block=32)
    want = ex.swiglu(g, u)
    near(h, want, (half + r8.silu_bound(g) + r8.U) * want.abs() + (u.abs() * (1 - g) + 1) * 2.0 ** -149 + zero, "h")
    q = bm.swiglu_rows8(gate, up, block=32)
    e = (r8.silu_bound(g) + r8.U) * want.abs() + (u.abs() * (1 - g) + 1) * 2.0 ** -149
    scale = r8.quantize(want, 32)[2]
    near(q.scale, scale, r8.blocks_of(e, 32).amax(2) / 127 + r8.U * scale + 2.0 ** -149, "scales")
    dg, du, h8 = bm.swiglu_checkpoint_backward(dh, g8, u8, need_h=True)
    gk, uk = (r8.values(x.codes.double(), x.scale.double(), 32) for x in (g8, u8))
    wg, wu = ex.swiglu_backward(d, gk, uk)
    wh = ex.swiglu(gk, uk)
    near(dg, wg, half * wg.abs() + r8.slope_bound(d, gk, uk) + ((d * uk).abs() + 1) * (1 - gk) * 2.0 ** -148 + zero, "dgate")
    near(du, wu, (half + r8.silu_bound(gk) + 3 * r8.U) * wu.abs() + (d.abs() * (1 - gk) + 1) * 2.0 ** -149 + zero, "dup")
    near(h8, wh, (half + r8.silu_bound(gk) + 3 * r8.U) * wh.abs() + (uk.abs() * (1 - gk) + 1) * 2.0 ** -149 + zero, "h again")
