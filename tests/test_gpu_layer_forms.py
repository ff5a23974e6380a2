"""The layer operators at sizes that reach every kernel form their plans
choose, against the plain 64-bit forms (tests/layers_forms.py has the sizes)."""

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
from layers_forms import FORMS  # noqa: E402

BF = torch.bfloat16


def sizes(op):
    return pytest.mark.parametrize("shape", FORMS[op], ids=["x".join(map(str, s)) for s in FORMS[op]])


def generator(m, n, k):
    return torch.Generator(device="cuda").manual_seed(3 * m + 5 * n + 7 * k)


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(BF)


def weight(gen, n, k):
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    w *= torch.exp(0.5 * torch.randn(n, 1, generator=gen, device="cuda"))
    return F.fp8_block_quantize(w)


@sizes("linear_act")
def test_linear_act(shape):
    m, n, k = shape
    gen = generator(*shape)
    x, (q, s), bias, residual = normal(gen, m, k), weight(gen, n, k), normal(gen, n), normal(gen, m, n)
    z = torch.empty(m, n, dtype=BF, device="cuda")
    say("linear_act", shape, "all of the epilogue")
    y = F.fp8_block_linear_act(x, q, s, bias=bias, residual=residual, act=F.ACT_GELU, z=z)
    torch.cuda.synchronize()
    R.check_linear_act(x, q, s, bias, residual, "gelu", y, z, f"{shape}")
    say("linear_act", shape, "plain")
    y = F.fp8_block_linear_act(x, q, s)
    torch.cuda.synchronize()
    R.check_linear_act(x, q, s, None, None, "none", y, None, f"{shape} plain")


@sizes("glu")
def test_glu(shape):
    m, n, k = shape
    gen = generator(*shape)
    x, (qg, sg), (qu, su) = normal(gen, m, k), weight(gen, n, k), weight(gen, n, k)
    g, u = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2))
    say("glu", shape, "kept")
    h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u)
    torch.cuda.synchronize()
    R.check_glu(x, qg, sg, qu, su, "silu", h, g, u, f"{shape}")
    say("glu", shape)
    h = F.fp8_block_glu(x, qg, sg, qu, su, act=F.ACT_GELU_TANH)
    torch.cuda.synchronize()
    R.check_glu(x, qg, sg, qu, su, "gelu_tanh", h, None, None, f"{shape}")


@sizes("linear_act_backward")
def test_linear_act_backward(shape):
    m, n, k = shape
    gen = generator(*shape)
    (q, s), dy, z = weight(gen, n, k), normal(gen, m, n), normal(gen, m, n, std=2.0)
    dbias = torch.empty(n, device="cuda")
    say("linear_act_backward", shape)
    dx, dz = F.fp8_block_linear_act_backward(dy, q, s, z=z, act=F.ACT_SILU, dbias=dbias)
    torch.cuda.synchronize()
    R.check_linear_act_backward(dy, z, q, s, "silu", dx, dz, dbias, f"{shape}")


@sizes("glu_backward")
def test_glu_backward(shape):
    m, n, k = shape
    gen = generator(*shape)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    dh, g, u = normal(gen, m, n), normal(gen, m, n, std=2.0), normal(gen, m, n)
    say("glu_backward", shape)
    dx, dg, du = F.fp8_block_glu_backward(dh, g, u, qg, sg, qu, su)
    torch.cuda.synchronize()
    R.check_glu_backward(dh, g, u, qg, sg, qu, su, "silu", dx, dg, du, f"{shape}")
