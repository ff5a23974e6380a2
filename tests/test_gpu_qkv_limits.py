"""From the QKV projection to its cache at the largest sizes there are: 2^31 - 1 tokens,
4096 heads of 256, 65536 tokens stored in a call; and the integer linear's 2^20
columns."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import int8_ref as I  # noqa: E402
import qkv_ref as R  # noqa: E402
from test_gpu_int8 import operands  # noqa: E402
from test_gpu_qkv import Case, cache, check_backward, check_forward, check_fused, check_store  # noqa: E402

BF = torch.bfloat16
T, D = 2 ** 31 - 1, 16
AT = torch.tensor([0, 1, 3, 2 ** 24 - 1, 2 ** 24, 2 ** 28 + 1, 2 ** 30, 2 ** 31 - 1027, 2 ** 31 - 6, 2 ** 31 - 3, 2 ** 31 - 2])


@pytest.fixture
def room():
    """200 GB of device memory, given back afterwards."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 210 << 30:
        pytest.skip("needs 210 GiB of free device memory")
    yield
    torch.cuda.empty_cache()


def nonzero(x):
    """Tokens with anything but zeros."""
    return sum(int((part.view(-1, D // 4).view(torch.int64) != 0).any(1).count_nonzero())
               for part in x.view(-1, D).view(torch.int64).split(1 << 27))


def one_head(values):
    """[T, 1, D] of zeros but for `values` at tokens AT."""
    x = torch.zeros(T, 1, D, dtype=BF, device="cuda")
    x[AT.cuda()] = values
    return x


def test_most_tokens(room):
    say("qk_norm_rope and its backward pass, tokens", T)
    c = Case(len(AT), 1, 1, D, 8)
    positions = torch.zeros(T, dtype=torch.int32, device="cuda")
    positions[AT.cuda()] = c.positions[0]
    q, none = one_head(c.q), torch.empty(T, 0, D, dtype=BF, device="cuda")
    table = (c.qw, c.kw, positions, c.freq)
    out, _ = F.fp8_qk_norm_rope(q, none, *table)
    small = F.fp8_qk_norm_rope(c.q, c.k[:, :0], *c.table)[0]
    assert torch.equal(out[AT.cuda()], small) and nonzero(out) == len(AT)
    del out
    dq = one_head(c.dq)
    dx, _, dw, _ = F.fp8_qk_norm_rope_backward(dq, none, q, none, *table, q_grad=dq, k_grad=none)
    ref = F.fp8_qk_norm_rope_backward(c.dq, c.k[:, :0], c.q, c.k[:, :0], *c.table)
    assert torch.equal(dx[AT.cuda()], ref[0]) and nonzero(dx) == len(AT)
    assert bool(((dw - ref[2]).abs() <= 2.0 ** -18 * ref[2].abs().amax()).all())


def test_most_tokens_read_back(room):
    say("kv_load, tokens", T)
    codes = cache(50, 1, D)
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[AT.cuda()] = torch.arange(len(AT), dtype=torch.int32, device="cuda") * 4
    k, v = F.fp8_kv_load(*codes, slots)
    small = slots[AT.cuda()]
    assert torch.equal(k[AT.cuda()], R.loaded(codes[0], codes[2], small))
    assert torch.equal(v[AT.cuda()], R.loaded(codes[1], codes[3], small))
    assert nonzero(k) == len(AT) and nonzero(v) == len(AT)


def test_most_heads():
    """4096 heads of 256: 16 MB a token and array."""
    t, h, d = 5, 4096, 256
    say("heads", h, d)
    c = Case(t, h, h, d, None, 3, False)
    check_forward(c, *F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how), (t, h, d))
    check_backward(c, F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how), (t, h, d))
    before = cache(t + 3, h, d)
    after = [x.clone() for x in before]
    slots = torch.tensor([7, 0, -1, 3, 0], dtype=torch.int32, device="cuda")
    q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how)
    check_fused(c, before, after, q, slots, (t, h, d))
    after = [x.clone() for x in before]
    F.fp8_kv_store(c.k, c.v, slots, *after)
    check_store(before, after, slots, R.stored(c.k), R.stored(c.v))
    k, v = F.fp8_kv_load(*after, slots)
    assert torch.equal(k, R.loaded(after[0], after[2], slots)) and torch.equal(v, R.loaded(after[1], after[3], slots))


@pytest.mark.parametrize("kind", ["random", "pages", "equal"])
def test_most_tokens_stored(kind):
    t, h, d = 65536, 2, 32
    say("kv_store, tokens", t, kind)
    c = Case(t, 1, h, d, 8)
    gen = torch.Generator().manual_seed(5)
    rows = t + 64
    slots = {"random": torch.randperm(rows, generator=gen)[:t],
             "pages": (torch.randperm(rows // 64, generator=gen)[:, None] * 64 + torch.arange(64)).reshape(-1)[:t],
             "equal": torch.randint(-3, rows // 3, (t,), generator=gen)}[kind].to(torch.int32).cuda()
    before = cache(rows, h, d)
    after = [x.clone() for x in before]
    F.fp8_kv_store(c.k, c.v, slots, *after)
    check_store(before, after, slots, R.stored(c.k), R.stored(c.v))
    after = [x.clone() for x in before]
    q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how)
    check_fused(c, before, after, q, slots, kind)


@pytest.mark.parametrize("m", [1, 20, 40, 300])
def test_most_columns(m):
    n, k = 2 ** 20, 80
    say("int8_linear", m, n, k)
    xq, xs, wq, ws, bias = operands(m, n, k)
    assert I.same_bits(F.int8_linear(xq, xs, wq, ws, bias=bias), I.linear(xq, xs, wq, ws, bias))
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(BF).cuda()
    assert I.same_bits(F.int8_linear_bf16(x, wq, ws, bias=bias), I.linear(*I.quantize(x), wq, ws, bias))
