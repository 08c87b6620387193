"""The float64 gradients that the GPU tests compare with, against central
differences of the forward formulas: the step h = 1e-5 leaves a truncation
error of order h^2 and a cancellation error of order 2^-53 / h, both below
1e-8 for values of order 1."""
import pytest
import torch

import _experts as ex

TOL = 1e-7


def _diff(f, a, h=1e-5):
    g = torch.zeros_like(a)
    flat, out = a.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        hi = f()
        flat[i] = keep - h
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * h)
    return g


def _rand(*shape, seed=0):
    return torch.randn(*shape, dtype=ex.F64, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_activation_slopes(name):
    z = _rand(4, 7, seed=1)
    d = _diff(lambda: ex.act(z, name).sum().item(), z)
    assert (d - ex.act_slope(z, name)).abs().max() < TOL


def test_expert_products():
    off = torch.tensor([0, 2, 2, 5])
    x, w, dy = _rand(5, 4, seed=2), _rand(3, 3, 4, seed=3), _rand(5, 3, seed=4)
    loss = lambda: (ex.expert_rows(x, w, off)[0] * dy).sum().item()  # noqa: E731
    assert (_diff(loss, x) - ex.expert_rows(dy, w, off, transposed=True)[0]).abs().max() < TOL
    assert (_diff(loss, w) - ex.expert_dw(dy, x, off)[0]).abs().max() < TOL


def test_swiglu_and_combine():
    g, u, d = _rand(3, 5, seed=5), _rand(3, 5, seed=6), _rand(3, 5, seed=7)
    dg, du = ex.swiglu_backward(d, g, u)
    loss = lambda: (ex.swiglu(g, u) * d).sum().item()  # noqa: E731
    assert (_diff(loss, g) - dg).abs().max() < TOL and (_diff(loss, u) - du).abs().max() < TOL
    o, w, dy = _rand(6, 4, seed=8), _rand(2, 3, seed=9), _rand(2, 4, seed=10)
    do, dw = ex.combine_backward(dy, o, w, 2, 3)
    loss = lambda: (ex.combine(o, w, 2, 3) * dy).sum().item()  # noqa: E731
    assert (_diff(loss, o) - do).abs().max() < TOL and (_diff(loss, w) - dw).abs().max() < TOL
