"""The layer operators' backward passes as a training step uses them: without
the input gradient, and inside autograd by the README's example."""

from __future__ import annotations

import os
import re

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


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(BF).cuda()


def weight(gen, n, k):
    return F.fp8_block_quantize((torch.randn(n, k, generator=gen) * 0.05).cuda())


@pytest.mark.parametrize("shape", [(1, 264, 512), (24, 1003, 272), (300, 264, 528)], ids=lambda s: "x".join(map(str, s)))
def test_without_the_input_gradient(shape):
    """need_dx=False gives None for dx and the same other gradients."""
    m, n, k = shape
    gen = torch.Generator().manual_seed(n)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    dy, z, u = normal(gen, m, n), normal(gen, m, n), normal(gen, m, n)
    d1, d2, d3 = (torch.empty(n, device="cuda") for _ in range(3))
    say("no input gradient", shape)
    _, dz = F.fp8_block_linear_act_backward(dy, qg, sg, z=z, act=F.ACT_GELU, dbias=d1)
    _, dg, du = F.fp8_block_glu_backward(dy, z, u, qg, sg, qu, su)
    none, dz2 = F.fp8_block_linear_act_backward(dy, qg, sg, z=z, act=F.ACT_GELU, dbias=d2, need_dx=False)
    none2, dg2, du2 = F.fp8_block_glu_backward(dy, z, u, qg, sg, qu, su, need_dx=False)
    none3, same = F.fp8_block_linear_act_backward(dy, qg, sg, dbias=d3, need_dx=False)
    torch.cuda.synchronize()
    assert none is None and none2 is None and none3 is None and same is dy
    assert torch.equal(dz, dz2) and torch.equal(d1, d2) and torch.equal(dg, dg2) and torch.equal(du, du2)
    total, size = dy.double().sum(0), dy.double().abs().sum(0)
    assert bool(((d3.double() - total).abs() <= R.sum_err(m, size) + R.TINY).all())
    with pytest.raises(ValueError):
        F.fp8_block_linear_act_backward(dy, qg, sg, dx=normal(gen, m, k), need_dx=False)
    with pytest.raises(ValueError):
        F.fp8_block_glu_backward(dy, z, u, qg, sg, qu, su, dx=normal(gen, m, k), need_dx=False)


def example(name):
    """The README's Python block that defines `name`."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), flags=re.S)
    space = {"torch": torch, "F": F}
    exec(next(b for b in blocks if f"class {name}(" in b), space)
    return space[name]


@pytest.mark.parametrize("m", [1, 40, 130])
def test_the_example_gives_the_gradient(m):
    """The autograd example between recorded operations: its gradient is the
    backward function's, that one the formula's in 64 bits, and the whole step
    runs twice with gradients that add up."""
    n, k = 264, 528
    gen = torch.Generator().manual_seed(m)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    x = normal(gen, m, k).requires_grad_(True)
    scale = normal(gen, n)
    say("autograd example", m)
    fn = example("FrozenGlu")
    h = fn.apply(x, qg, sg, qu, su)
    (h * scale).sum().backward()
    first = x.grad.clone()
    (fn.apply(x, qg, sg, qu, su) * scale).sum().backward()
    with torch.no_grad():
        g, u = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2))
        want_h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u)
        dh = scale.expand(m, n).contiguous()
        dx, dg, du = F.fp8_block_glu_backward(dh, g, u, qg, sg, qu, su)
    torch.cuda.synchronize()
    assert torch.equal(h.detach(), want_h) and torch.equal(first, dx) and torch.equal(x.grad, dx + dx)
    R.check_glu(x.detach(), qg, sg, qu, su, "silu", want_h, g, u, "example")
    R.check_glu_backward(dh, g, u, qg, sg, qu, su, "silu", dx, dg, du, "example")
    with pytest.raises(RuntimeError, match="not recorded by autograd"):
        F.fp8_block_glu(x, qg, sg, qu, su)
