"""The feed-forward block's gradient bound (tests/layers_block.py) on the CPU:
the 64-bit gradient against differences, the operators' roundings inside the
bound, and wrong gradients outside."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import layers_block as B  # noqa: E402
from layers_ref import act64, grad64  # noqa: E402

BF = torch.bfloat16


def block(m, hidden=384, inner=784):
    gen = torch.Generator().manual_seed(m)
    rows = lambda n, k: (torch.randn(n, k, generator=gen) * 0.05 *                     # noqa: E731
                         torch.exp(0.5 * torch.randn(n, 1, generator=gen))).to(BF).double()
    wg, wu, wd = rows(inner, hidden), rows(inner, hidden), rows(hidden, inner)
    x, dy = (torch.randn(m, hidden, generator=gen).to(BF).double() for _ in range(2))
    return x, dy, wg, wu, wd


def rounded(t):
    return t.to(BF).double()


def operators(x, dy, wg, wu, wd):
    """The gradient with the operators' roundings: its two terms and dy."""
    g, u, dh = rounded(x @ wg.t()), rounded(x @ wu.t()), rounded(dy @ wd)
    return rounded(dh * u * grad64(g, "silu")) @ wg, rounded(dh * act64(g, "silu")) @ wu, dy


@pytest.mark.parametrize("m", [1, 24])
def test_gradient_against_differences(m):
    x, dy, wg, wu, wd = block(m)
    want, _ = B.gradient64(x, dy, wg, wu, wd)
    gen = torch.Generator().manual_seed(1)
    for _ in range(4):
        v = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        diff = float((B.loss64(x + h * v, dy, wg, wu, wd) - B.loss64(x - h * v, dy, wg, wu, wd)) / (2 * h))
        # central differences are off by h^2 times a third derivative
        assert abs(diff - float((want * v).sum())) <= 1e-6 * float((want * v).abs().sum())


@pytest.mark.parametrize("m", [1, 24, 200])
def test_bound_takes_the_roundings_and_nothing_else(m):
    args = block(m)
    gate, up, dy = operators(*args)
    whole = lambda *terms: rounded(rounded(sum(terms[:-1])) + terms[-1])               # noqa: E731
    assert B.worst(whole(gate, up, dy), *args) <= 1.0
    zero = torch.zeros_like(gate)
    wrong = {"nothing": zero, "negated": -whole(gate, up, dy), "no gate term": whole(zero, up, dy),
             "no up term": whole(gate, zero, dy), "no residual": whole(gate, up, zero),
             "residual twice": whole(gate, up, 2 * dy), "a tenth more": 1.1 * whole(gate, up, dy),
             "gate term negated": whole(-gate, up, dy), "last row of zeros": None}
    last = whole(gate, up, dy).clone()
    last[-1] = 0
    wrong["last row of zeros"] = last
    for name, got in wrong.items():
        assert B.worst(got, *args) > 1.5, (name, B.worst(got, *args))
