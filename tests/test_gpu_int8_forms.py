"""The forms of the 8-bit integer linear that tests/test_gpu_int8.py does not run
(tests/int8_forms.py), bit for bit; and the single row that is quantized on the way
between guards, captured, and with values that are not finite."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import int8_ref as R  # noqa: E402
from int8_forms import CODES, FROM_BF16  # noqa: E402
from test_gpu_int8 import operands  # noqa: E402

BF = torch.bfloat16


def ids(shapes):
    return ["x".join(map(str, s)) for s in shapes]


def row_of(m, k, seed=0):
    gen = torch.Generator().manual_seed(k + seed)
    x = torch.randn(m, k, generator=gen) * torch.exp(torch.randn(m, 1, generator=gen))
    x[:, 3::97] *= 4
    return x.to(BF).cuda()


@pytest.mark.parametrize("shape", CODES, ids=ids(CODES))
def test_from_codes(shape):
    say("int8_linear", *shape)
    xq, xs, wq, ws, bias = operands(*shape)
    assert R.same_bits(F.int8_linear(xq, xs, wq, ws, bias=bias), R.linear(xq, xs, wq, ws, bias))
    assert R.same_bits(F.int8_linear(xq, xs, wq, ws), R.linear(xq, xs, wq, ws))


@pytest.mark.parametrize("shape", FROM_BF16, ids=ids(FROM_BF16))
def test_from_bf16(shape):
    """The definition's bits, and those of the two calls."""
    say("int8_linear_bf16", *shape)
    m, n, k = shape
    _, _, wq, ws, bias = operands(m, n, k)
    x = row_of(m, k)
    codes = R.quantize(x)
    for b in (None, bias):
        y = F.int8_linear_bf16(x, wq, ws, bias=b)
        assert R.same_bits(y, R.linear(*codes, wq, ws, b))
        assert R.same_bits(y, F.int8_linear(*F.int8_row_quantize(x), wq, ws, bias=b))


@pytest.mark.parametrize("kind", ["zeros", "subnormal", "largest", "ties", "one"])
@pytest.mark.parametrize("n", [4100, 40])
def test_special_rows_quantized_on_the_way(kind, n):
    k = 528
    _, _, wq, ws, bias = operands(1, n, k)
    x = {"zeros": torch.zeros(k), "subnormal": (torch.arange(k) % 191 - 95) * 2.0 ** -133,
         "largest": torch.where(torch.arange(k) % 2 == 0, 1.0, -1.0) * torch.finfo(BF).max,
         "ties": (torch.arange(k) % 255 - 127) * 0.5, "one": torch.eye(k)[77]}[kind].to(BF)[None].cuda()
    if kind == "ties":
        x[0, 0] = 127.0                    # scale 1: every odd half is a tie
    y = F.int8_linear_bf16(x, wq, ws, bias=bias)
    assert R.same_bits(y, R.linear(*R.quantize(x), wq, ws, bias))


@pytest.mark.parametrize("shape", [(1, 4101, 528), (1, 8000, 8192)])
def test_writes_only_its_output(shape):
    """A row of odd length between guards, the workspace full of NaNs and left alone."""
    m, n, k = shape
    _, _, wq, ws, bias = operands(m, n, k)
    x = row_of(m, k)
    size = F.int8_workspace_size(m, n, k)
    buf = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((n + 256,), 3.0, dtype=BF, device="cuda")
    y = out[128:128 + n].view(m, n)
    F.int8_linear_bf16(x, wq, ws, bias=bias, out=y, workspace=buf[256:256 + size])
    assert R.same_bits(y, R.linear(*R.quantize(x), wq, ws, bias))
    assert bool((out[:128] == 3).all()) and bool((out[128 + n:] == 3).all())
    assert bool((buf[:256] == 0xFF).all()) and bool((buf[256 + size:] == 0xFF).all())


@pytest.mark.parametrize("shape", [(1, 4101, 528), (1, 8000, 8192)])
def test_captured_and_replayed(shape):
    m, n, k = shape
    _, _, wq, ws, bias = operands(m, n, k)
    x = torch.zeros(m, k, dtype=BF, device="cuda")
    y = torch.empty(m, n, dtype=BF, device="cuda")
    work = torch.empty(F.int8_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(torch.cuda.Stream()):
        F.int8_linear_bf16(x, wq, ws, bias=bias, out=y, workspace=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.int8_linear_bf16(x, wq, ws, bias=bias, out=y, workspace=work)
    for i in range(4):
        x.copy_(row_of(m, k, i))
        graph.replay()
        torch.cuda.synchronize()
        assert R.same_bits(y, R.linear(*R.quantize(x), wq, ws, bias))
        work.fill_(0xFF)
        torch.cuda.synchronize()
