"""The activations where they are small: relative precision, in each kernel
that evaluates them (the streams' epilogue, the tiles' and the join's).

Room, relative to the 64-bit value: the half step of bf16, and of the value
before it is rounded

* GELU, -12 <= t < 0: the tail Phi(-a) is off by 6.0e-7 for its polynomial in
  fp32, a^2 2^-24 for its exponent's rounding, and one unit each (2^-23) for
  the hardware's exp2 and reciprocal and the product with t: below
  6.0e-7 + a^2 2^-24 + 3 2^-23, 1e-5 at a = 12.
* SiLU and the tanh GELU, down to v = -80: (2 |v| + 4) 2^-23 for the sigmoid,
  one more unit for the product with t. Its v is a polynomial in fp32: three
  roundings and two rounded constants, inside the 2 |v|.

The bias holds t and the product is zero, so the kernels see t exactly."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
from layers_ref import HALF  # noqa: E402

BF = torch.bfloat16
UNIT = 2.0 ** -23


def gelu(t):
    # (torch's ndtr is (1 + erf) / 2, which is 0 below t = -8.3)
    return 0.5 * t * torch.special.erfc(-t * math.sqrt(0.5)), 6.0e-7 + t * t * 2.0 ** -24 + 3 * UNIT


def silu(t):
    return t / (1 + torch.exp(-t)), (2 * t.abs() + 5) * UNIT


def gelu_tanh(t):
    v = 2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)
    return t / (1 + torch.exp(-v)), (2 * v.abs() + 5) * UNIT


ACTS = {"gelu": (F.ACT_GELU, gelu, 12.0), "silu": (F.ACT_SILU, silu, 80.0), "gelu_tanh": (F.ACT_GELU_TANH, gelu_tanh, 9.5)}
# rows, K: a stream, a stream with K splits and the join, tiles, tiles with K
# splits and the join
WAYS = {"stream": (1, 16), "stream split": (1, 8192), "tiles": (40, 16), "tiles split": (40, 8192)}


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("act", list(ACTS))
def test_small_values_keep_their_precision(act, way):
    number, form, lowest = ACTS[act]
    m, k = WAYS[way]
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    t = bits[(bits.float() >= -lowest) & (bits.float() <= -2.0 ** -10)].cuda()
    t = t[: t.numel() // 4 * 4].contiguous()
    n = t.numel()
    assert n > 1500
    assert (F.layer_workspace_size("linear_act", m, n, k) > 0) == ("split" in way)
    x = torch.zeros(m, k, dtype=BF, device="cuda")
    q = torch.zeros(n, k, dtype=torch.uint8, device="cuda")
    s = torch.ones(F.scale_grid_shape(n, k), device="cuda")
    say("activation", act, way, n)
    y = F.fp8_block_linear_act(x, q, s, bias=t, act=number)
    torch.cuda.synchronize()
    want, error = form(t.double())
    off = (y.double() - want).abs() / want.abs()
    room = HALF * (1 + error) + error
    assert bool((off <= room).all()), float((off / room).max())
    # that a value is there at all is part of it: a lost tail is off by 1
    assert bool((y.float() < 0).all())
