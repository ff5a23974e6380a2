"""The 8-bit integer linear by its definition, step by step: whole sums in 64
bits, and the fp32 roundings that the interface names one by one, so that every
output bit is determined."""

from __future__ import annotations

import torch


def fp32(x: torch.Tensor) -> torch.Tensor:
    """fl32 of a value computed in fp64. Rounding a quotient, product or sum of
    fp32 values to fp64 first does not change its fp32 rounding (53 >= 2 * 24 + 2)."""
    return x.to(torch.float32)


def quantize(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes int8 [M,K], scales fp32 [M])."""
    x = x.double()
    s = fp32(x.abs().amax(1) / 127.0)
    s[s == 0] = 1.0
    t = fp32(x / s.double()[:, None]).double()
    return t.round().clamp(-127, 127).to(torch.int8), s


def linear(xq, xs, wq, ws, bias=None) -> torch.Tensor:
    """bf16 y: the sum in fp64 (whole numbers below 2^53: exact)."""
    acc = fp32(xq.double() @ wq.double().t()).double()
    scale = fp32(xs.double()[:, None] * ws.double()[None]).double()
    y = fp32(acc * scale)
    if bias is not None:
        y = fp32(y.double() + bias.double())
    return y.to(torch.bfloat16)


def same_bits(a: torch.Tensor, b: torch.Tensor) -> bool:
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.dtype == b.dtype and a.shape == b.shape and bool((a.contiguous().view(kind) == b.contiguous().view(kind)).all())
