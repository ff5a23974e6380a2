"""The 8-bit integer linear at the most rows there are, 2^31 - 1 of them."""

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

BF = torch.bfloat16
M, N, K = 2 ** 31 - 1, 1, 16
# rows next to the tiles' edges at both ends, and to 2^25 (a quantizer's launch)
ROWS = torch.tensor([0, 1, 63, 64, 255, 256, 2 ** 25 - 1, 2 ** 25, 2 ** 30, 2 ** 31 - 513, 2 ** 31 - 258, 2 ** 31 - 257,
                     2 ** 31 - 256, 2 ** 31 - 129, 2 ** 31 - 128, 2 ** 31 - 65, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 3,
                     2 ** 31 - 2])


@pytest.fixture
def room():
    """130 GB of device memory, given back afterwards."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 140 << 30:
        pytest.skip("needs 140 GiB of free device memory")
    yield
    torch.cuda.empty_cache()


def others_are(y, value):
    """Every row but ROWS is `value`."""
    at = ROWS.cuda()
    kept = y[at].clone()
    y[at] = value
    same = all(bool((part == value).all()) for part in y.view(-1).split(1 << 28))
    y[at] = kept
    return same


def test_codes(room):
    say("int8_linear", M, N, K)
    gen = torch.Generator().manual_seed(1)
    xq = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    xs = torch.ones(M, device="cuda")
    at = ROWS.cuda()
    xq[at] = torch.randint(-128, 128, (len(at), K), generator=gen, dtype=torch.int8).cuda()
    xs[at] = (torch.rand(len(at), generator=gen) + 0.5).cuda()
    wq = torch.randint(-128, 128, (N, K), generator=gen, dtype=torch.int8).cuda()
    ws, bias = torch.full((N,), 0.25, device="cuda"), torch.full((N,), 1.5, dtype=BF, device="cuda")
    y = F.int8_linear(xq, xs, wq, ws, bias=bias)
    assert R.same_bits(y[at], R.linear(xq[at], xs[at], wq, ws, bias))
    assert others_are(y, 1.5)


def test_from_bf16(room):
    say("int8_linear_bf16", M, N, K)
    gen = torch.Generator().manual_seed(2)
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    at = ROWS.cuda()
    x[at] = torch.randn(len(at), K, generator=gen).to(BF).cuda()
    wq = torch.randint(-128, 128, (N, K), generator=gen, dtype=torch.int8).cuda()
    ws, bias = torch.full((N,), 0.25, device="cuda"), torch.full((N,), 1.5, dtype=BF, device="cuda")
    y = F.int8_linear_bf16(x, wq, ws, bias=bias)
    assert R.same_bits(y[at], R.linear(*R.quantize(x[at]), wq, ws, bias))
    assert others_are(y, 1.5)
