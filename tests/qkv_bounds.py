"""How far norm, rotation and their gradients may be from the definitions in 64 bits, by
what the kernels do (tests/qkv_ref.py derives wider bounds, for coarser angles).

With u = 2^-24 and half a bf16 step 2^-8 of the value:
  r: squares of bf16 are exact in fp32; a lane's eight take 7 roundings, the sum over
    at most 32 lanes 5; the division by D (its reciprocal and the product) 2, eps and
    the sum with it 2: the mean is off by 16 u, its root by 8 u, and the reciprocal root
    itself by one step, 2 u: 10 u;
  a factor: the angle is exact to 2^-53, sine and cosine to 2e-10 and one rounding of a
    number below 1, u / 2: 0.51 u in all (absolute);
  an output r fma(x, w c, xo (wo s)): w c and wo s one rounding each on the factors'
    own, one of xo's product, the fma's, r's and its product's: of |a| + |b|, with a and
    b the pair after the norm, 0.51 + 1 + 1 + 1 + 10 + 1 < 15 u;
  dn = fma(y, c, -(o s)): 0.51 + 1 + 1 < 3 u of |a| + |b| of the gradient's pair; with
    the weight 4 u;
  mean(u x): 4 u, the fma's of 8 values, 5 sums, two for D: 19 u of the terms' sizes;
    along = mean r r: two of r's 10 u and 2 roundings, 41 u in all;
  dx = r fma(-x, along, u): (4 + 1) u of u, (41 + 1) u of x along, and r's 10 u and its
    product 1: 16 u of r |u|, 53 u of r |x| r^2 mean |u x|;
  dw, a sum of dn r x: 3 u, r's 10, one rounding of dn r: 14 u of a term, and a
    rounding for each of the sums a term goes through.
Heads out of the scaled range are scaled by a power of two, which rounds nothing."""

from __future__ import annotations

import torch

import qkv_angles as A
import qkv_ref as R

U = 2.0 ** -24


def normed(x, eps):
    return (x.square().mean(-1, keepdim=True) + eps).rsqrt()


def forward(x, w, cos, sin, eps, interleaved):
    """(out, bound before the bf16 rounding), both fp64."""
    x, w = x.double(), w.double()
    n = x * normed(x, eps) * w
    size, _ = R.reach(n, cos, interleaved)
    return A.turn(n, cos, sin, interleaved), 15 * U * size


def backward(dy, x, w, cos, sin, eps, interleaved, steps):
    """(dx, its bound before the bf16 rounding, dw, its bound). `steps`: the most terms
    of dw that one lane adds in a row."""
    dy, x, w = dy.double(), x.double(), w.double()
    r = normed(x, eps)
    dn = A.turn(dy, cos, -sin, interleaved)
    size, _ = R.reach(dy, cos, interleaved)
    u = dn * w
    dx = r * (u - x * r.square() * (u * x).mean(-1, keepdim=True))
    along = r.square() * (size * w.abs() * x.abs()).mean(-1, keepdim=True)
    bound = r * U * (16 * size * w.abs() + 53 * x.abs() * along)
    dw = (dn * x * r).sum((0, 1))
    # a lane's terms, then at most 5 + 4 + 16 + 6 sums
    return dx, bound, dw, ((14 + steps + 31) * U * size * x.abs() * r).sum((0, 1))
