"""The layer operators at the ends of what their header allows: n and k of
2^20, and the arrays that need no more than 4-byte alignment (scale grids and
dbias) at such an address."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import layers_ref as R  # noqa: E402

BF = torch.bfloat16
MOST = 1 << 20


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(BF)


def weight(gen, n, k):
    """A weight whose scale grid starts 4 bytes past a 16-byte boundary."""
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    w *= torch.exp(0.5 * torch.randn(n, 1, generator=gen, device="cuda"))
    q, s = F.fp8_block_quantize(w)
    return q, off_by_four(s)


def off_by_four(t):
    buf = torch.full((t.numel() + 2,), float("nan"), device="cuda")
    view = buf[1:1 + t.numel()].view(t.shape)
    view.copy_(t)
    assert view.data_ptr() % 16 == 4
    return view


SHAPES = [(3, MOST, 16), (40, MOST, 16), (300, MOST - 3, 16), (3, 16, MOST), (24, 24, MOST), (40, 24, MOST), (300, 7, MOST),
          # ordinary sizes, for the alignment
          (1, 264, 512), (20, 1003, 272), (77, 1003, 656), (300, 264, 528), (2048, 8448, 4096)]


@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_limits(shape):
    m, n, k = shape
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    x, (qg, sg), (qu, su) = normal(gen, m, k), weight(gen, n, k), weight(gen, n, k)
    bias, residual = normal(gen, n), normal(gen, m, n)
    z, g, u = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(3))
    say("limits, linear_act", shape)
    y = F.fp8_block_linear_act(x, qg, sg, bias=bias, residual=residual, act=F.ACT_SILU, z=z)
    torch.cuda.synchronize()
    R.check_linear_act(x, qg, sg, bias, residual, "silu", y, z, f"{shape}")
    say("limits, glu", shape)
    h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u)
    torch.cuda.synchronize()
    R.check_glu(x, qg, sg, qu, su, "silu", h, g, u, f"{shape}")
    del y, h, z
    dy = normal(gen, m, n)
    dbias = off_by_four(torch.zeros(n, device="cuda"))
    say("limits, linear_act_backward", shape)
    dx, dz = F.fp8_block_linear_act_backward(dy, qg, sg, z=g, act=F.ACT_GELU, dbias=dbias)
    torch.cuda.synchronize()
    R.check_linear_act_backward(dy, g, qg, sg, "gelu", dx, dz, dbias, f"{shape}")
    say("limits, glu_backward", shape)
    dx, dg, du = F.fp8_block_glu_backward(dy, g, u, qg, sg, qu, su)
    torch.cuda.synchronize()
    R.check_glu_backward(dy, g, u, qg, sg, qu, su, "silu", dx, dg, du, f"{shape}")
