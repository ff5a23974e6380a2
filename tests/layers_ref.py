"""Plain 64-bit forms of the layer operators and the error bounds of the
kernels, used by the layer tests.

Bounds, per output element (bf16 half step: 2^-8 of the value; A = the same
product over absolute values):

* a fp32 sum of R exact bf16 products, in any order: each of the R additions
  is off by at most one unit of a partial sum of size at most A:
  (R + 8) 2^-23 A (a whole unit, so that truncating adders are covered; the
  8 stand for the joins of split sums).
* an activation evaluated at t: 2^-20 |t|. A sigmoid on exp2 and a reciprocal
  is off by a relative (|v| + 4) 2^-23 of p(v), and |v| p(-|v|) < 0.37, so
  t p is off by at most 4.4 * 2^-23 |t|; erfc's few units give the same.
* its derivative: 2^-20 (1 + |t|), by the same count on p (1 + t (1 - p)).
* slopes: |act'| <= 1.13 for every activation here.

Where the kernels evaluate otherwise than counted above they stay inside: a
sigmoid off by (2 |v| + 4) 2^-23 (fp8bl_act.h) makes t p off by at most 4.8 *
2^-23 |t|, and the GELU's tail polynomial, which stands where erfc did, is off
by a relative 6.0e-7 + a^2 2^-24 + 3 * 2^-23 of Phi(-a) <= 1/2: at most
5 * 2^-23 |t|.
"""

from __future__ import annotations

import math

import torch

import block_scaled_fp8_linear_amd as F

HALF = 2.0 ** -8
EVAL = 2.0 ** -20
SLOPE = 1.13
TINY = 1e-36          # outputs below the normal range of bf16
ACTS = {"none": F.ACT_NONE, "relu": F.ACT_RELU, "silu": F.ACT_SILU, "gelu": F.ACT_GELU,
        "gelu_tanh": F.ACT_GELU_TANH}


def sum_err(r: int, a: torch.Tensor) -> torch.Tensor:
    return (r + 8) * 2.0 ** -23 * a


def act64(t: torch.Tensor, act: str) -> torch.Tensor:
    if act == "none":
        return t
    if act == "relu":
        return torch.where(t > 0, t, torch.zeros_like(t))
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return t * torch.special.ndtr(t)
    return 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))


def grad64(t: torch.Tensor, act: str) -> torch.Tensor:
    if act == "none":
        return torch.ones_like(t)
    if act == "relu":
        return (t > 0).double()
    if act == "silu":
        p = 1 / (1 + torch.exp(-t))
        return p * (1 + t * (1 - p))
    if act == "gelu":
        return torch.special.ndtr(t) + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)
    a, b = math.sqrt(2 / math.pi), 0.044715
    h = torch.tanh(a * (t + b * t ** 3))
    return 0.5 * (1 + h) + 0.5 * t * (1 - h * h) * a * (1 + 3 * b * t * t)


def weight64(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    """W^ in 64 bits: the code times its block's scale in fp32, then bf16."""
    n, k = q.shape
    wide = s.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return (q.view(torch.float8_e4m3fn).float() * wide).to(torch.bfloat16).double()


def within(got: torch.Tensor, want: torch.Tensor, err: torch.Tensor, what: str) -> float:
    """got (bf16, rounded from a value within err of want) against want."""
    off = (got.double() - want).abs()
    room = HALF * (want.abs() + err) + err + TINY
    worst = float((off / room).max()) if off.numel() else 0.0
    assert not math.isnan(worst) and worst <= 1.0, (what, worst)
    return worst


def check_linear_act(x, q, s, bias, residual, act, y, z, what=""):
    w, xd = weight64(q, s), x.double()
    zr = xd @ w.t()
    err = sum_err(x.shape[1], xd.abs() @ w.abs().t())
    if bias is not None:
        zr = zr + bias.double()
        err = err + 2.0 ** -23 * zr.abs()
    if z is not None:
        within(z, zr, err, what + " z")
    yr = act64(zr, act)
    err = SLOPE * err + EVAL * zr.abs()
    if residual is not None:
        yr = yr + residual.double()
        err = err + 2.0 ** -23 * yr.abs()
    return within(y, yr, err, what + " y")


def check_linear_act_backward(dy, z, q, s, act, dx, dz, dbias, what=""):
    d = dy.double()
    err = torch.zeros_like(d)
    if act != "none":
        t = z.double()
        err = d.abs() * EVAL * (1 + t.abs())
        d = d * grad64(t, act)
        within(dz, d, err, what + " dz")
    if dbias is not None:
        off = (dbias.double() - d.sum(0)).abs()
        room = err.sum(0) + sum_err(dy.shape[0], d.abs().sum(0)) + TINY
        assert bool((off <= room).all()), (what, "dbias", float((off / room).max()))
    # the product reads the dz it returned
    w, e = weight64(q, s), dz.double()
    return within(dx, e @ w, sum_err(dy.shape[1], e.abs() @ w.abs()), what + " dx")


def check_glu(x, qg, sg, qu, su, act, h, g, u, what=""):
    wg, wu, xd = weight64(qg, sg), weight64(qu, su), x.double()
    gr, ur = xd @ wg.t(), xd @ wu.t()
    eg = sum_err(x.shape[1], xd.abs() @ wg.abs().t())
    eu = sum_err(x.shape[1], xd.abs() @ wu.abs().t())
    if g is not None:
        within(g, gr, eg, what + " g")
        within(u, ur, eu, what + " u")
    ar = act64(gr, act)
    ea = SLOPE * eg + EVAL * gr.abs()
    return within(h, ar * ur, ea * (ur.abs() + eu) + ar.abs() * eu + 2.0 ** -23 * (ar * ur).abs(), what + " h")


def check_glu_backward(dh, g, u, qg, sg, qu, su, act, dx, dg, du, what=""):
    d, t, v = dh.double(), g.double(), u.double()
    within(dg, d * v * grad64(t, act), (d * v).abs() * EVAL * (1 + t.abs()), what + " dg")
    within(du, d * act64(t, act), d.abs() * EVAL * t.abs(), what + " du")
    wg, wu, eg, eu = weight64(qg, sg), weight64(qu, su), dg.double(), du.double()
    return within(dx, eg @ wg + eu @ wu,
                  sum_err(2 * dh.shape[1], eg.abs() @ wg.abs() + eu.abs() @ wu.abs()), what + " dx")
