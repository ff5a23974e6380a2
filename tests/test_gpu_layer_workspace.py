"""The layer operators with a workspace of exactly the queried size, full of
NaNs, between sentinels: what they read of it they wrote, and they write
nothing beside it."""

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
FENCE, MARK = 1 << 16, 0x5A


class Workspace:
    def __init__(self, op, m, n, k):
        self.size = F.layer_workspace_size(op, m, n, k)
        assert self.size > 0, (op, m, n, k)
        self.all = torch.full((self.size + 2 * FENCE,), MARK, dtype=torch.uint8, device="cuda")
        self.view = self.all[FENCE:FENCE + self.size]
        assert self.view.data_ptr() % 256 == 0
        self.view.fill_(0xFF)          # a NaN in fp32 and in bf16

    def kept(self):
        return bool((self.all[:FENCE] == MARK).all()) and bool((self.all[FENCE + self.size:] == MARK).all())


def generator(m, n, k):
    return torch.Generator(device="cuda").manual_seed(m + n + k)


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(BF)


def weight(gen, n, k):
    return F.fp8_block_quantize(torch.randn(n, k, generator=gen, device="cuda") * 0.02)


# streams and each tile with K splits, rows of quads and odd ones, and columns
# left over (the last three, two of them with odd rows)
FORWARD = [(4, 72, 4368), (24, 1003, 16384), (40, 1000, 5120), (77, 1003, 5120), (512, 1443, 5120),
           (512, 5121, 25600), (2048, 8448, 4096), (2048, 9001, 2048), (3000, 2819, 1552)]


@pytest.mark.parametrize("shape", FORWARD, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape):
    m, n, k = shape
    gen = generator(*shape)
    x, (qg, sg), (qu, su) = normal(gen, m, k), weight(gen, n, k), weight(gen, n, k)
    bias, res = normal(gen, n), normal(gen, m, n)
    z, g, u = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(3))
    ran = 0
    if F.layer_workspace_size("linear_act", *shape):
        ws = Workspace("linear_act", *shape)
        say("workspace, linear_act", shape, ws.size)
        y = F.fp8_block_linear_act(x, qg, sg, bias=bias, residual=res, act=F.ACT_SILU, z=z, workspace=ws.view)
        torch.cuda.synchronize()
        R.check_linear_act(x, qg, sg, bias, res, "silu", y, z, f"{shape}")
        assert ws.kept()
        ran += 1
    if F.layer_workspace_size("glu", *shape):
        ws = Workspace("glu", *shape)
        say("workspace, glu", shape, ws.size)
        h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u, workspace=ws.view)
        torch.cuda.synchronize()
        R.check_glu(x, qg, sg, qu, su, "silu", h, g, u, f"{shape}")
        assert ws.kept()
        ran += 1
    assert ran


# padded gradients (N no multiple of 8), column sums of several chunks (more
# than 256 rows) and split partials, together and one by one
BACKWARD = [(16, 264, 1040), (24, 1003, 2064), (77, 1003, 656), (300, 1003, 656), (300, 5121, 1040), (513, 1443, 336),
            (700, 2819, 400), (1500, 2819, 12288), (2048, 4099, 8448)]


@pytest.mark.parametrize("shape", BACKWARD, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape):
    m, n, k = shape
    gen = generator(*shape)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    dy, z, u = normal(gen, m, n), normal(gen, m, n, std=2.0), normal(gen, m, n)
    dbias = torch.empty(n, device="cuda")
    ws = Workspace("linear_act_backward", *shape)
    say("workspace, linear_act_backward", shape, ws.size)
    dx, dz = F.fp8_block_linear_act_backward(dy, qg, sg, z=z, act=F.ACT_GELU, dbias=dbias, workspace=ws.view)
    torch.cuda.synchronize()
    R.check_linear_act_backward(dy, z, qg, sg, "gelu", dx, dz, dbias, f"{shape}")
    assert ws.kept()
    ws.view.fill_(0xFF)
    say("workspace, linear_act_backward without an activation", shape)
    dx, _ = F.fp8_block_linear_act_backward(dy, qg, sg, dbias=dbias, workspace=ws.view)
    torch.cuda.synchronize()
    R.check_linear_act_backward(dy, None, qg, sg, "none", dx, dy, dbias, f"{shape} none")
    assert ws.kept()
    ws = Workspace("glu_backward", *shape)
    say("workspace, glu_backward", shape, ws.size)
    dx, dg, du = F.fp8_block_glu_backward(dy, z, u, qg, sg, qu, su, workspace=ws.view)
    torch.cuda.synchronize()
    R.check_glu_backward(dy, z, u, qg, sg, qu, su, "silu", dx, dg, du, f"{shape}")
    assert ws.kept()
