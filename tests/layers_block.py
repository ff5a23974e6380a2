"""A feed-forward block on the layer operators,

    y = (silu(x Wg^T) * (x Wu^T)) Wd^T + x,

its input gradient in 64 bits, and how far the operators' gradient may be from
it.

The operators round to bf16 what they keep or hand on: g, u, dh, dg, du and dx,
and the caller's sum dx + dy. A rounding is off by a relative e with |e| <= d =
2^-8. Those of g, u, dh, dg and du reach an element of dx as a sum of terms c e,
one for each of the inner columns and arrays, with c the derivative of dx by
the logarithm of the rounded value (first order; the second is 2^-8 smaller).
Errors of different elements are as good as independent and have mean zero, so
a sum of many is bounded as such sums are (Hoeffding): uniform errors in
[-d, d] have variance d^2 / 3, V = d^2 / 3 sum c^2, and the sum passes
7 sqrt(V) with a probability below 2 e^(-24.5) = 5e-11, over the 77000 elements
of the largest case below 4e-6. To that come the last two roundings in full
(a half step of dx and one of dx + dy), a tenth for what is of second order,
and the fp32 sums: (R + 8) 2^-23 of the sum over absolute values, twice, one
for dh and one for dx.

With 784 inner columns that is 3 to 5% of the gradient's size: far less than
any of its terms."""

from __future__ import annotations

import torch

from layers_ref import HALF, act64, grad64, sum_err


def curve64(t: torch.Tensor) -> torch.Tensor:
    """silu''(t)."""
    p = 1 / (1 + torch.exp(-t))
    return p * (1 - p) * (2 + t * (1 - 2 * p))


def loss64(x, dy, wg, wu, wd):
    """sum(y dy) of the block in 64 bits."""
    return ((act64(x @ wg.t(), "silu") * (x @ wu.t())) @ wd.t() + x).mul(dy).sum()


def gradient64(x, dy, wg, wu, wd):
    """(the input gradient, its room) in 64 bits; all arguments are doubles."""
    g, u, dh = x @ wg.t(), x @ wu.t(), dy @ wd
    a, a1, a2 = act64(g, "silu"), grad64(g, "silu"), curve64(g)
    dg, du = dh * u * a1, dh * a
    dx = dg @ wg + du @ wu
    gg, uu, gu = wg * wg, wu * wu, wg * wu

    def squares(p, q):           # sum over the inner columns of (p Wg + q Wu)^2
        return p.square() @ gg + 2 * (p * q) @ gu + q.square() @ uu

    v = squares(dg, du)                                      # dh
    v = v + squares(dh * g * u * a2, dh * g * a1)            # g
    v = v + 2 * dg.square() @ gg + du.square() @ uu          # u, dg; du
    v = v.clamp_min(0) * HALF ** 2 / 3
    size = dg.abs() @ wg.abs() + du.abs() @ wu.abs()
    sums = sum_err(wd.shape[0], (dy.abs() @ wd.abs()) * (u * a1).abs()) @ wg.abs() \
        + sum_err(wd.shape[0], (dy.abs() @ wd.abs()) * a.abs()) @ wu.abs() \
        + sum_err(2 * wg.shape[0], size)
    room = 1.1 * (7 * v.sqrt() + HALF * dx.abs() + HALF * (dx + dy).abs()) + sums
    return dx + dy, room


def worst(got, x, dy, wg, wu, wd) -> float:
    """The largest part of its room that an element of `got` is off by."""
    want, room = gradient64(x, dy, wg, wu, wd)
    return float(((got.double() - want).abs() / room).max())
