"""The oracle of the operators in 8 bits and of the block norms: what the codes
have to hold, and the norms' gradients against automatic ones and differences."""
import pytest
import torch

import _experts as ex
import _rows8 as r8


@pytest.mark.parametrize("C,block", [(1, 0), (7, 0), (200, 0), (64, 32), (100, 64), (129, 128), (31, 32)])
def test_codes_hold_the_rows(C, block):
    x = torch.randn(9, C, generator=torch.Generator().manual_seed(C), dtype=ex.F64)
    x[3] = 0
    _, q, scale = r8.quantize(x, block)
    assert q.abs().max() <= 127 and (q == q.round()).all() and (q[3] == 0).all() and (scale[3] == 0).all()
    v = r8.values(q, scale[:, 0] if not block else scale, block)
    wide = scale.repeat_interleave(block or C, 1)[:, :C]
    assert ((v - x).abs() <= wide / 2 * (1 + 1e-12)).all()
    most = r8.blocks_of(q.abs(), block).amax(2)
    assert (most[[0, 1, 2, 4, 5, 6, 7, 8]] == 127).all()                    # the largest of a block keeps its value


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_quotients_of_16_bit_values_are_ties_or_far_from_them(dtype):
    """What lets float32 find the codes of 64 bits: 127 x / m of 16-bit x and m is
    a tie exactly, or further from one than float32's rounding of a quotient."""
    g = torch.Generator().manual_seed(1)
    m = torch.rand(400, 1, generator=g).add(0.5).to(dtype).double()
    x = torch.cat([m * torch.rand(400, 300, generator=g).double(), m / 2, m / 254, m / 127], 1).to(dtype).double()
    x = torch.minimum(x, m)
    t = 127 * x / m
    off = (t - t.floor() - 0.5).abs()
    exact = (254 * x) / m % 2 == 1
    assert exact[:, 300].all()                                              # m / 2 is the tie 63.5
    assert (off[~exact] > 4 * t[~exact] * 2.0 ** -24).all()


def case(T, H, seed, gate_rows):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=ex.F64)  # noqa: E731
    return rnd(T, H), rnd(T, H), rnd(H) + 1, rnd(*gate_rows), rnd(H) + 1, rnd(T, H), rnd(T, H)


@pytest.mark.parametrize("gate_rows", [(6,), (5, 6)])
def test_block_norm_gradients(gate_rows):
    o, r, wa, gate, wb, ds, dn = case(5, 6, 3, gate_rows)
    scale, eps = 0.7, 1e-3
    leaves = [t.clone().requires_grad_() for t in (o, r, wa, gate, wb)]

    def f(o, r, wa, gate, wb):
        return r8.block_norm(o, r, wa, gate, scale, wb, eps)
    s, n = f(*leaves)
    auto = torch.autograd.grad([s, n], leaves, [ds, dn])
    d_o, dres, dwa, dg, dwb = r8.block_norm_backward(dn, ds, s.detach(), o, wa, gate, scale, wb, eps)
    for got, want in zip((d_o, dres, dwa, dg.sum(0) if len(gate_rows) == 1 else dg, dwb), auto):
        assert torch.allclose(got, want, rtol=1e-10, atol=1e-12)
    # and differences of the formula itself, one direction each
    for i, (x, grad) in enumerate(zip((o, r, wa, gate, wb), auto)):
        d = torch.randn(x.shape, generator=torch.Generator().manual_seed(i), dtype=ex.F64)
        h = 1e-5
        args = [[y + (sign * h * d if j == i else 0) for j, y in enumerate((o, r, wa, gate, wb))] for sign in (1, -1)]
        (s1, n1), (s0, n0) = f(*args[0]), f(*args[1])
        diff = (((s1 - s0) * ds).sum() + ((n1 - n0) * dn).sum()) / (2 * h)
        assert abs(diff - (grad * d).sum()) <= 1e-7 * (1 + abs(diff))


def test_bounds_are_what_float32_needs():
    """The formulas evaluated in float32 stay inside their bounds (and not by much
    more than the sums' worst case allows)."""
    o, r, wa, gate, wb, ds, dn = case(40, 300, 4, (300,))
    F = torch.float32
    f32 = [t.float() for t in (o, r, wa, gate, wb)]
    args64 = [t.double() for t in f32]
    s, n, es, en = r8.norm_bounds(args64[0], args64[1], args64[2], args64[3], 0.7, args64[4], 1e-6, F, F)
    s32, n32 = r8.block_norm(f32[0], f32[1], f32[2], f32[3], 0.7, f32[4], 1e-6)
    assert ((s32.double() - s).abs() <= es).all() and ((n32.double() - n).abs() <= en).all()
    ds, dn = ds.float(), dn.float()
    back = lambda c, s: r8.block_norm_backward(c(dn), c(ds), c(s), *(c(t) for t in f32[:1]), c(f32[2]), c(f32[3]), 0.7, c(f32[4]), 1e-6)  # noqa: E731
    got = back(lambda t: t, s32)
    want, bounds = r8.norm_backward_bounds(dn.double(), ds.double(), s32.double(), args64[0], args64[2], args64[3], 0.7,
                                           args64[4], 1e-6, F, F, F)
    for x, name in zip(got, ("d_o", "dresidual", "dw_after", "dgate", "dw_before")):
        assert ((x.double() - want[name]).abs() <= bounds[name]).all(), name
