"""A feed-forward block forward and backward through the layer operators,
against the block's gradient in 64 bits (tests/layers_block.py has the bound,
tests/test_layers_block_cpu.py shows what it rejects)."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import layers_block as B  # noqa: E402
import layers_ref as R  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("m", [1, 24, 200])
def test_block_gradient(m):
    hidden, inner = 384, 784
    gen = torch.Generator().manual_seed(m)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).to(BF).cuda()

    def weight(n, k):
        w = torch.randn(n, k, generator=gen) * 0.05 * torch.exp(0.5 * torch.randn(n, 1, generator=gen))
        return F.fp8_block_quantize(w.cuda())

    (qg, sg), (qu, su), (qd, sd) = weight(inner, hidden), weight(inner, hidden), weight(hidden, inner)
    x, dy = normal(m, hidden), normal(m, hidden)
    g, u = (torch.empty(m, inner, dtype=BF, device="cuda") for _ in range(2))
    say("block gradient", m)
    h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u)
    y = F.fp8_block_linear_act(h, qd, sd, residual=x)
    dh, _ = F.fp8_block_linear_act_backward(dy, qd, sd)
    dx, dg, du = F.fp8_block_glu_backward(dh, g, u, qg, sg, qu, su)
    torch.cuda.synchronize()
    # each step on what it was given
    R.check_glu(x, qg, sg, qu, su, "silu", h, g, u, "block")
    R.check_linear_act(h, qd, sd, None, x, "none", y, None, "block")
    R.check_linear_act_backward(dy, None, qd, sd, "none", dh, dy, None, "block")
    R.check_glu_backward(dh, g, u, qg, sg, qu, su, "silu", dx, dg, du, "block")
    # and the whole
    worst = B.worst(dx + dy, x.double(), dy.double(), R.weight64(qg, sg), R.weight64(qu, su), R.weight64(qd, sd))
    say("block gradient", m, "off by", round(worst, 3), "of the bound")
    assert worst <= 1.0
