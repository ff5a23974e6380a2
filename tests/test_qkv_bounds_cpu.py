"""The bounds of tests/qkv_bounds.py hold for the kernels' arithmetic done step by step
in fp32, and reject factors from a coarser angle."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import qkv_angles as A  # noqa: E402
import qkv_bounds as B  # noqa: E402
import qkv_ref as R  # noqa: E402

BF = torch.bfloat16


def case(interleaved, t=60, h=6, d=64):
    gen = torch.Generator().manual_seed(7 + interleaved)
    x, dy = (torch.randn(t, h, d, generator=gen).to(BF) for _ in range(2))
    w = (1 + 0.3 * torch.randn(d, generator=gen)).to(BF)
    positions = torch.randint(0, 1000, (1, t), generator=gen, dtype=torch.int32)
    freq = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float()
    return x, dy, w, positions, freq


def rounded(x, w, cos, sin, interleaved):
    """A head as the forward kernel works it out, every step rounded to fp32."""
    x, w, cos, sin = x.float(), w.float(), cos.float(), sin.float()
    r = torch.rsqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
    i, p = torch.arange(cos.shape[-1]), cos.shape[-1]
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + p)
    out = torch.empty_like(x)
    out[..., a] = r * (x[..., a] * (w[a] * cos) - x[..., b] * (w[b] * sin))
    out[..., b] = r * (x[..., b] * (w[b] * cos) + x[..., a] * (w[a] * sin))
    return out


@pytest.mark.parametrize("interleaved", [False, True])
def test_fp32_steps_are_inside(interleaved):
    x, _, w, positions, freq = case(interleaved)
    cos, sin = A.turns(positions, freq, None)
    ref, bound = B.forward(x, w, cos, sin, 1e-6, interleaved)
    assert bool(((rounded(x, w, cos, sin, interleaved).double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_an_fp32_angle_is_rejected(interleaved):
    """As bf16 results, and the same for the gradients."""
    x, dy, w, positions, freq = case(interleaved)
    cos, sin = A.turns(positions, freq, None)
    theta = (positions[0].float()[:, None, None] * freq).double()        # the product rounded to fp32
    for name, angle in (("product", theta), ("turns", (theta / 6.283185307179586).float().double() * 6.283185307179586)):
        c, s = angle.cos(), angle.sin()
        ref, bound = B.forward(x, w, cos, sin, 1e-6, interleaved)
        right, wrong = rounded(x, w, cos, sin, interleaved), rounded(x, w, c, s, interleaved)
        assert R.outside(right.to(BF), ref, bound) <= 1
        assert R.outside(wrong.to(BF), ref, bound) > 1, name
        dx, db, dw, dwb = B.backward(dy, x, w, cos, sin, 1e-6, interleaved, 1)
        other = B.backward(dy, x, w, c, s, 1e-6, interleaved, 1)
        assert R.outside(dx.to(BF), dx, db) <= 1 and R.outside(other[0].to(BF), dx, db) > 1, name


def test_the_bounds_are_tighter():
    x, dy, w, positions, freq = case(False)
    cos, sin = A.turns(positions, freq, None)
    ref, bound = B.forward(x, w, cos, sin, 1e-6, False)
    wide_ref, wide = R.forward(x, w, positions, freq, None, 1e-6, False)
    assert float((ref - wide_ref).abs().max()) < 1e-9 and bool((bound <= wide / 3).all())
    dx, db, dw, dwb = B.backward(dy, x, w, cos, sin, 1e-6, False, 3)
    wide = R.backward(dy, x, w, positions, freq, None, 1e-6, False, 3)
    assert float((dx - wide[0]).abs().max()) < 1e-9 and bool((db <= wide[1] / 3).all()) and bool((dwb < wide[3]).all())
