"""Norm, rotation and the E4M3 cache by their definitions in 64 bits, and how far
an fp32 evaluation may be from them.

Bounds, with u = 2^-24 (fp32) and half a bf16 step 2^-8 of the value:
  r = (mean x^2 + eps)^-1/2: a sum of D products and D roundings is off by at
    most (D + 2) u relative, r by half of that and 2 u for the root;
  theta: in fp64 as turns, off by 2^-51 |theta| after two products; its
    fraction is rounded to fp32 (2^-25 turns, 2^-22.3 rad) and the sine and
    cosine are good to 2^-22, so each factor is off by 2^-21 + 2^-51 |theta|;
  an output a c - b s: products, sum and the weight's products add 6 u.
  Together (|a| + |b|) ((D / 2 + 3 + 6) u + 8 u + 2^-51 |theta|) <=
    (|a| + |b|) ((D / 2 + 24) u + 2^-51 |theta|), and 2^-8 |out| for bf16."""

from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def members(pairs: int, interleaved: bool) -> tuple[torch.Tensor, torch.Tensor]:
    i = torch.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def angles(positions, inv_freq, axes) -> torch.Tensor:
    """theta [T, 1, P]."""
    positions = positions.view(-1, positions.shape[-1]).double()
    which = torch.zeros(inv_freq.numel(), dtype=torch.long) if axes is None else torch.tensor(list(axes))
    return (positions[which.to(positions.device)] * inv_freq.double()[:, None]).t()[:, None]


def turn(x, theta, interleaved):
    a, b = members(theta.shape[-1], interleaved)
    out = x.clone()
    c, s = theta.cos(), theta.sin()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def reach(x, theta, interleaved):
    """|a| + |b| of each element's pair, |x| for those that are not turned, and
    |theta| likewise (0)."""
    a, b = members(theta.shape[-1], interleaved)
    size, far = x.abs().clone(), torch.zeros_like(x)
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    far[..., a] = far[..., b] = theta.abs().expand(x.shape[0], x.shape[1], -1)
    return size, far


def forward(x, w, positions, inv_freq, axes, eps, interleaved):
    """(out, bound before the bf16 rounding), both fp64."""
    x, theta = x.double(), angles(positions, inv_freq, axes)
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    size, far = reach(n, theta, interleaved)
    return turn(n, theta, interleaved), size * ((x.shape[-1] / 2 + 24) * U + 2.0 ** -51 * far)


def backward(dy, x, w, positions, inv_freq, axes, eps, interleaved, steps):
    """(dx, its bound before the bf16 rounding, dw, its bound). `steps`: the most
    terms of dw that one lane adds in a row."""
    dy, x, w, theta = dy.double(), x.double(), w.double(), angles(positions, inv_freq, axes)
    d = x.shape[-1]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    dn = turn(dy, -theta, interleaved)
    size, far = reach(dy, theta, interleaved)
    u = dn * w
    dx = r * (u - x * r.square() * (u * x).mean(-1, keepdim=True))
    # |u| is at most size |w|: every factor and sum as above, D roundings in the
    # mean of u x on top
    each = (2 * d + 48) * U + 2.0 ** -51 * far
    along = r.square() * (size * w.abs() * x.abs() * each).mean(-1, keepdim=True)
    bound = r * (size * w.abs() * each + x.abs() * along)
    dw = (dn * x * r).sum((0, 1))
    # a lane's sum of `steps` terms, then at most 5 + 4 + 16 + 6 sums
    dw_bound = (size * x.abs() * r * ((d / 2 + 32 + steps + 31) * U + 2.0 ** -51 * far)).sum((0, 1))
    return dx, bound, dw, dw_bound


def outside(got, ref, bound) -> float:
    """The largest |got - ref| over what it may be (1 at the bound) for bf16."""
    got = got.double()
    assert bool(torch.isfinite(got).all())
    return float(((got - ref).abs() / (HALF_BF16 * ref.abs() + bound + 1e-38)).max()) if got.numel() else 0.0


# ---- the cache ----------------------------------------------------------

def _values() -> torch.Tensor:
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append(-x if c >= 128 else x)
    return torch.tensor(v, dtype=torch.float64)


VALUES = _values()


def values(codes: torch.Tensor) -> torch.Tensor:
    return VALUES.to(codes.device)[codes.long()]


def scales(x: torch.Tensor) -> torch.Tensor:
    """fl32(max|x| / 448) of each head, 1 where that is 0."""
    s = (x.double().abs().amax(-1) / 448.0).to(torch.float32)
    return torch.where(s == 0, torch.ones_like(s), s)


def nearest(x: torch.Tensor) -> torch.Tensor:
    """x to the nearest E4M3 value, ties to the even code, at most 448."""
    _, e = torch.frexp(x)
    step = (((e - 4).clamp_min(-9).long() + 1023) << 52).view(torch.float64)     # 2^(e - 4), from its bits
    return ((x / step).round() * step).clamp(-448, 448)


def stored(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(E4M3 values fp64, scales fp32) of bf16 or fp32 heads."""
    s = scales(x)
    return nearest((x.double() / s.double()[..., None]).to(torch.float32).double()), s


def stored_turned(x, w, positions, inv_freq, axes, eps, interleaved):
    """(E4M3 values, scales, where the values are sure, where the scales are) of the
    fused store's keys: sure where fp64's own error cannot cross a border."""
    ref, _ = forward(x, w, positions, inv_freq, axes, eps, interleaved)
    n = x.double() / (x.double().square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    size, far = reach(n, angles(positions, inv_freq, axes), interleaved)
    off = size * (2.0 ** -38 + 2.0 ** -50 * far)
    top, most, s = ref.abs().amax(-1), off.amax(-1), scales(ref)
    sure = ((top - most) / 448.0).to(torch.float32) == ((top + most) / 448.0).to(torch.float32)

    def code(z):
        return nearest((z / s.double()[..., None]).to(torch.float32).double())

    return code(ref), s, (code(ref - off) == code(ref + off)) & sure[..., None], sure


def loaded(codes, scale, slots) -> torch.Tensor:
    """bf16 rows, zeros for a slot outside the cache."""
    kept = (slots >= 0) & (slots < codes.shape[0])
    rows = torch.where(kept, slots, torch.zeros_like(slots)).long()
    x = (values(codes[rows]) * scale[rows].double()[..., None]).to(torch.float32).to(torch.bfloat16)
    return torch.where(kept[:, None, None], x, torch.zeros_like(x))


def last_ones(slots, rows: int) -> torch.Tensor:
    """Which tokens are stored: in the cache, and no later one has the slot."""
    seen, live = set(), []
    for s in reversed(slots.tolist()):
        live.append(0 <= s < rows and s not in seen)
        seen.add(s)
    return torch.tensor(live[::-1], dtype=torch.bool)
