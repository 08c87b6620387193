"""Rows in 8 bits on the GPU against float64: codes equal, values within their
roundings; the gated activation into them and with its inputs kept in them.
Bounds: _rows8.py."""
import pytest

import _experts as ex
import _rows8 as r8
from _gpu import require_gpu, say, torch
from test_gpu_experts import BF, F32, HF, check, gen, place, rnd

pytestmark = pytest.mark.gpu
BLOCKS = (0, 32, 64, 128)


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def bm():
    import bit_moe_amd
    return bit_moe_amd


def out_rows8(bm, R, C, block, pad=0, shift=0):
    """A Rows8 whose rows lie apart, all bytes 77 and scales 5 before the call."""
    codes = place(torch.full((R, C), 77, dtype=torch.int8), pad, shift, hold=77)
    n = -(-C // block) if block else 1
    scale = place(torch.full((R, n), 5.0), pad, hold=5.0)
    return bm.Rows8(codes, scale if block else scale[:, 0], block)


def scales(q):
    """[R, blocks] in float64."""
    s = q.scale.cpu().double()
    return s if q.block else s[:, None]


SHAPES = [(1, 1, 0, 0), (3, 7, 0, 0), (5, 100, 3, 1), (2, 512, 0, 0), (1100, 520, 0, 0), (1030, 1001, 1, 3), (4, 2049, 0, 0),
          (1025, 2050, 0, 0), (3, 7168, 16, 16), (1026, 7168, 0, 0), (6, 9000, 5, 0), (2, 40000, 0, 0), (17, 128, 0, 0),
          (300, 33, 0, 5), (1024, 4104, 0, 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("block", BLOCKS)
def test_quantize_rows(bm, shape, dtype, block):
    R, C, pad, shift = shape
    g = gen(R + C + block)
    x, x64 = rnd(g, R, C, dtype=dtype, pad=pad, shift=shift)
    say(f"[rows8] quantize {shape} {dtype} block {block}")
    q = out_rows8(bm, R, C, block, pad, shift)
    assert bm.quantize_rows(x, block=block, out=q) is q
    t, codes, scale = r8.quantize(x64, block)
    got = q.codes.cpu().double()
    if dtype is F32:                        # a quotient next to a tie may go either way: off by its own rounding
        assert ((got - t).abs() <= 0.5 + 127 * 2 * r8.U).all()
    else:
        assert torch.equal(got, codes)
    check(scales(q), scale, r8.U * scale, "scales")
    if pad and R > 1:                       # nothing between the rows
        assert (q.codes.as_strided((R - 1, pad), (C + pad, 1), shift + C) == 77).all()
    new = bm.quantize_rows(x, block=block)
    assert torch.equal(new.codes, q.codes) and torch.equal(new.scale, q.scale)
    for to in (BF, HF, F32):
        v = r8.values(got, scales(q) if block else scales(q)[:, 0], block)
        y = place(torch.full((R, C), 7.0, dtype=to), pad, shift, hold=3.0)
        bm.dequantize_rows(q, y=y)
        check(y, v, ex.half_ulp(to) * (1 + r8.U) * v.abs() + (r8.U * v.abs() if to is not F32 else 0) + 2.0 ** -25 * (to is HF),
              f"values in {to}")
        assert torch.equal(bm.dequantize_rows(q, dtype=to), y)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "fp16", "fp32"])
def test_quantize_special_values(bm, block, dtype):
    """Zeros, ties, infinities, NaN, the type's largest and smallest values, each in
    a row of its own and beside ordinary blocks."""
    C = 300
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x = torch.randn(12, C, generator=gen(5)).to(dtype)
    x[0] = 0
    x[1, :] = 0
    x[1, 40] = 1.0
    x[1, 41], x[1, 42] = 0.5, -0.5                      # 63.5: to the even 64
    x[2, 7] = float("inf")
    x[3, 290] = float("nan")
    x[4, 100] = float("-inf")
    x[5] = (torch.rand(C, generator=gen(6)) * 2 - 1) * big
    x[5, 0] = -big
    x[6] = torch.randn(C, generator=gen(7)) * tiny * 300
    x[7, :] = -0.0
    x[8, :] = big
    x[9, :] = tiny
    x[10, :] = 0
    x[10, 299] = tiny
    say(f"[rows8] special values {dtype} block {block}")
    q = bm.quantize_rows(x.cuda(), block=block)
    got, sc = q.codes.cpu().double(), scales(q)
    x64 = x.double()
    b = r8.blocks_of(x64, block)
    bad = ~torch.isfinite(b).all(2)
    assert torch.equal(torch.isnan(sc), bad)
    wide_bad = bad.repeat_interleave(b.shape[2], 1)[:, :C]
    assert (got[wide_bad] == 0).all()
    t, codes, scale = r8.quantize(torch.where(wide_bad, 0, x64), block)
    if dtype is F32:
        assert ((got - t)[~wide_bad].abs() <= 0.5 + 127 * 2 * r8.U).all()
    else:
        assert torch.equal(got[~wide_bad], codes[~wide_bad])
    assert got[1, 41] == (64 if 40 // (block or C) == 41 // (block or C) else 127)
    ok = ~bad
    # float32's largest value / 127 lies nearer to the float above it, 127 times which is
    # infinite: the one below is taken, up to a whole step (2^-23) off, not half a one
    step = torch.where(127 * scale == torch.finfo(F32).max, 2, 1) * r8.U
    assert ((sc - scale).abs() <= step * scale + 2.0 ** -150)[ok].all()
    y = bm.dequantize_rows(q, dtype=F32).cpu().double()
    assert torch.isnan(y[wide_bad]).all() and torch.isfinite(y[~wide_bad]).all()


def test_quantize_experts_and_no_rows(bm):
    w = torch.randn(3, 10, 48, generator=gen(1)).to(BF).cuda()
    q = bm.quantize_rows(w)
    flat = bm.quantize_rows(w.view(30, 48))
    assert torch.equal(q.codes.view(30, 48), flat.codes) and torch.equal(q.scale.view(30), flat.scale)
    assert q.codes.shape == (3, 10, 48) and q.scale.shape == (3, 10)
    with pytest.raises(ValueError):
        bm.quantize_rows(w[:, :5])
    assert bm.quantize_rows(w[:, :5].contiguous()).codes.shape == (3, 5, 48)
    none = bm.quantize_rows(w.view(30, 48)[:0], block=32)
    assert none.codes.shape == (0, 48) and bm.dequantize_rows(none).shape == (0, 48)


@pytest.mark.parametrize("R,I,pad,shift", [(1, 2048, 0, 0), (8, 1, 0, 0), (37, 100, 4, 1), (1030, 520, 0, 0), (3, 9000, 0, 0),
                                           (2, 33000, 0, 0), (1100, 2048, 0, 0), (5, 2056, 8, 8), (70, 300, 0, 0)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("block", BLOCKS)
def test_swiglu_rows8(bm, R, I, pad, shift, dtype, block):
    g = gen(R + I)
    z, z64 = rnd(g, R, 2 * I, dtype=dtype, scale=2.0, pad=pad, shift=shift)
    gate, up = z64[:, :I], z64[:, I:]
    say(f"[rows8] swiglu_rows8 R={R} I={I} {dtype} block {block}")
    q = out_rows8(bm, R, I, block, pad, shift)
    bm.swiglu_rows8(z[:, :I], z[:, I:], block=block, out=q)
    h = ex.swiglu(gate, up)
    e = (r8.silu_bound(gate) + r8.U) * h.abs()
    _, _, scale = r8.quantize(h, block)
    # m's error is at most the block's largest; the codes then hold the float32 h
    es = r8.blocks_of(e, block).amax(2) / 127 + r8.U * scale
    check(scales(q), scale, es, "scales")
    v = r8.values(q.codes.cpu().double(), scales(q) if block else scales(q)[:, 0], block)
    wide = scales(q).repeat_interleave(block or I, 1)[:, :I]
    check(v, h, wide * (0.5 + 127 * 3 * r8.U) + e, "values")
    new = bm.swiglu_rows8(z[:, :I], z[:, I:], block=block)
    assert torch.equal(new.codes, q.codes) and torch.equal(new.scale, q.scale)


@pytest.mark.parametrize("R,I,pad,shift", [(1, 2048, 0, 0), (8, 1, 0, 0), (37, 100, 4, 1), (300, 520, 0, 0), (5, 2056, 8, 8),
                                           (9, 31, 0, 0), (64, 257, 0, 0), (2, 7168, 0, 0)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("block", BLOCKS[1:])
def test_swiglu_checkpoint(bm, R, I, pad, shift, dtype, block):
    g = gen(R + I + 1)
    z, z64 = rnd(g, R, 2 * I, dtype=dtype, scale=2.0, pad=pad, shift=shift)
    dh, d64 = rnd(g, R, I, dtype=dtype, pad=pad, shift=shift)
    gate, up = z[:, :I], z[:, I:]
    say(f"[rows8] checkpoint R={R} I={I} {dtype} block {block}")
    h, g8, u8 = bm.swiglu_checkpoint(gate, up, block=block)
    want = ex.swiglu(z64[:, :I], z64[:, I:])
    small = 2.0 ** -25 * (dtype is HF)
    u = ex.half_ulp(dtype) * (1 + 2.0 ** -8)
    check(h, want, (u + r8.silu_bound(z64[:, :I]) + r8.U) * want.abs() + small, "h")
    for got, x in ((g8, gate), (u8, up)):                       # as quantize_rows gives them
        q = bm.quantize_rows(x, block=block)
        assert got.block == block and torch.equal(got.codes, q.codes) and torch.equal(got.scale, q.scale)
    # into given ones, apart from each other
    to = [out_rows8(bm, R, I, block, pad, shift) for _ in range(2)]
    h2, a, b = bm.swiglu_checkpoint(gate, up, block=block, h=place(torch.zeros(R, I, dtype=dtype), pad, shift),
                                    gate8=to[0], up8=to[1])
    assert a is to[0] and torch.equal(h2, h) and torch.equal(a.codes, g8.codes) and torch.equal(b.scale, u8.scale)
    # the backward pass, at the kept values
    gk, uk = (r8.values(q.codes.cpu().double(), scales(q), block) for q in (g8, u8))
    dg, du, h8 = bm.swiglu_checkpoint_backward(dh, g8, u8, need_h=True)
    wg, wu = ex.swiglu_backward(d64, gk, uk)
    wh = ex.swiglu(gk, uk)
    check(dg, wg, u * wg.abs() + r8.slope_bound(d64, gk, uk) + small, "dgate")
    check(du, wu, (u + r8.silu_bound(gk) + 3 * r8.U) * wu.abs() + small, "dup")
    check(h8, wh, (u + r8.silu_bound(gk) + 3 * r8.U) * wh.abs() + small, "h again")
    dg2, du2, none = bm.swiglu_checkpoint_backward(dh, a, b)
    assert none is None and torch.equal(dg2, dg) and torch.equal(du2, du)
    # over dh itself
    d2 = dh.clone()
    _, du3, _ = bm.swiglu_checkpoint_backward(d2, g8, u8, dgate=d2, dup=torch.empty_like(dh))
    assert torch.equal(d2, dg) and torch.equal(du3, du)
    d2 = dh.clone()
    bm.swiglu_checkpoint_backward(d2, g8, u8, dgate=torch.empty_like(dh), dup=d2)
    assert torch.equal(d2, du)


def test_checkpoint_gradients_against_differences(bm):
    """dgate and dup are the slopes of swiglu at the kept values: central
    differences of the float64 formula in a random direction."""
    z = torch.randn(40, 2 * 96, generator=gen(3)).to(BF)
    dh = torch.randn(40, 96, generator=gen(4)).to(BF)
    _, g8, u8 = bm.swiglu_checkpoint(z[:, :96].cuda(), z[:, 96:].cuda(), block=32)
    dg, du, _ = bm.swiglu_checkpoint_backward(dh.cuda(), g8, u8)
    g, u = (r8.values(q.codes.cpu().double(), q.scale.cpu().double(), 32) for q in (g8, u8))
    a, b = torch.randn(2, 40, 96, generator=gen(5), dtype=ex.F64)
    step = 1e-5
    f = lambda t: (ex.swiglu(g + t * a, u + t * b) * dh.double()).sum()  # noqa: E731
    diff = (f(step) - f(-step)) / (2 * step)
    got = (dg.cpu().double() * a).sum() + (du.cpu().double() * b).sum()
    # each gradient's rounding and float32 error, and the difference's own third-order term
    wg, wu = ex.swiglu_backward(dh.double(), g, u)
    slack = (ex.half_ulp(BF) * (1 + 2.0 ** -8) * (wg.abs() * a.abs() + wu.abs() * b.abs()) + r8.slope_bound(dh.double(), g, u) * a.abs() +
             r8.silu_bound(g) * wu.abs() * b.abs()).sum() + 1e-6 * (1 + abs(diff))
    assert abs(diff - got) <= slack


def test_long_rows_past_32_bits(bm):
    """Rows whose elements lie beyond 2^32 bytes of the matrix's start."""
    R, C, ld = 5, 2048, (1 << 30) + 64
    say("[rows8] rows 2 GiB apart")
    x = torch.empty(R * ld, dtype=BF, device="cuda").as_strided((R, C), (ld, 1))
    v = torch.randn(R, C, generator=gen(9)).to(BF)
    x.copy_(v)
    codes = torch.empty(R * ld, dtype=torch.int8, device="cuda").as_strided((R, C), (ld, 1))
    for block in (0, 64):
        q = bm.Rows8(codes, torch.empty((R, 32) if block else R, device="cuda"), block)
        bm.quantize_rows(x, block=block, out=q)
        _, want, scale = r8.quantize(v.double(), block)
        assert torch.equal(q.codes.cpu().double(), want)
        bm.dequantize_rows(q, y=x)
        y = r8.values(want, scale if block else scale[:, 0], block)
        check(x, y, (ex.half_ulp(BF) + 4 * r8.U) * y.abs(), "back")
        x.copy_(v)
