"""The sine and cosine of position * inv_freq at any position, by whole numbers: the
product is a fraction with a power of two below it, and turns are taken off it with
pi to 60 digits, so that what fp64 gets is the exact angle's rest rounded once."""

from __future__ import annotations

import math

import torch

# pi / 2 as a multiple of 2^-SHIFT
SHIFT = 180
DIGITS = "314159265358979323846264338327950288419716939937510582097494"
HALF_PI = (int(DIGITS) << SHIFT) // (2 * 10 ** (len(DIGITS) - 1))


def rest(position: int, inv_freq: float) -> tuple[int, float]:
    """(quarter turns, the angle behind them within pi / 4)."""
    num, den = inv_freq.as_integer_ratio()
    theta = (position * num << SHIFT) // den
    quarters = (2 * theta + HALF_PI) // (2 * HALF_PI)
    return quarters % 4, math.ldexp(float(theta - quarters * HALF_PI), -SHIFT)


def turns(positions: torch.Tensor, inv_freq: torch.Tensor, axes) -> tuple[torch.Tensor, torch.Tensor]:
    """cos and sin [T, 1, P] in fp64 of positions [axes, T] and fp32 inv_freq [P]."""
    rows, freq = positions.cpu().tolist(), inv_freq.cpu().tolist()
    which = list(axes) if axes is not None else [0] * len(freq)
    cos, sin = [], []
    for t in range(len(rows[0])):
        for a, f in zip(which, freq):
            q, r = rest(rows[a][t], f)
            c, s = math.cos(r), math.sin(r)
            cos.append((c, -s, -c, s)[q])
            sin.append((s, c, -s, -c)[q])
    shape = (len(rows[0]), 1, len(freq))
    return (torch.tensor(x, dtype=torch.float64).view(shape).to(positions.device) for x in (cos, sin))


def turn(x, cos, sin, interleaved):
    """x [T, H, D] fp64 with its pairs turned."""
    p = cos.shape[-1]
    i = torch.arange(p)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + p)
    out = x.clone()
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out
