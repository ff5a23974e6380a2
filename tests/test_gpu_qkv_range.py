"""Norm and rotation of heads whose squares, or whose eps, leave the range of fp32:
subnormal heads and the largest ones, an eps of 0, below fp32 and far above the
squares, heads of zeros. The definitions and bounds are those of tests/qkv_ref.py;
a head of zeros with an eps of 0 is zeros by the interface."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import qkv_ref as R  # noqa: E402
from test_gpu_qkv import Case, cache  # noqa: E402

BF = torch.bfloat16

# The power of two that each head is scaled by: below and above fp32's squares, next
# to the borders of the range that needs no scale, and ordinary ones between them.
POWERS = (-80, 0, -133, 100, -16, 32, -120, 1, 120, -17, 33, -60)
EPS = (0.0, 1e-300, 1e-50, 1e-30, 1e-12, 1e-6, 1e30)
SIZES = [(9, 6, 2, 64, None, 3, False), (7, 3, 5, 80, 16, 1, True), (5, 2, 3, 16, 8, 1, False), (3, 9, 2, 256, None, 2, True)]
IDS = ["-".join(map(str, s[:4])) for s in SIZES]


def scaled(x):
    """Each head of x by a power of two of its own, every seventh head zeros."""
    t, h = x.shape[:2]
    i = torch.arange(t * h, device="cuda").view(t, h)
    by = torch.tensor(POWERS, device="cuda")[i % len(POWERS)]
    x = torch.ldexp(x.double().clamp(-8, 8), by[..., None]).to(BF)
    x[i % 7 == 3] = 0
    return x.contiguous()


def case(size):
    c = Case(*size)
    c.q, c.k = scaled(c.q), scaled(c.k)
    return c


def substitute(x, eps):
    """x with ones in the place of heads of zeros where eps is 0, and where those are."""
    empty = (x == 0).all(-1, keepdim=True) & (eps == 0)
    return torch.where(empty, torch.ones_like(x), x), empty


def forward(c, x, w, eps):
    filled, empty = substitute(x, eps)
    ref, bound = c.ref(filled, w, eps)
    return torch.where(empty, 0.0, ref), torch.where(empty, 0.0, bound)


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_norm_rope(size, eps):
    say("qk_norm_rope", size, eps)
    c = case(size)
    q, k = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how, eps=eps)
    for got, x, w in ((q, c.q, c.qw), (k, c.k, c.kw)):
        worst = R.outside(got, *forward(c, x, w, eps))
        assert worst <= 1, worst


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_backward(size, eps):
    """Where the gradient itself is past bf16's largest value it is infinite."""
    say("qk_norm_rope_backward", size, eps)
    c = case(size)
    got = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how, eps=eps)
    most = torch.finfo(BF).max
    for dx, dw, dy, x, w in ((got[0], got[2], c.dq, c.q, c.qw), (got[1], got[3], c.dk, c.k, c.kw)):
        filled, empty = substitute(x, eps)
        dy = torch.where(empty, torch.zeros_like(dy), dy)
        ref, bound, wref, wbound = c.ref_back(dy, filled, w, eps)
        past = ref.abs() >= most * (1 + 2.0 ** -9) + bound
        held = ref.abs() < most * (1 - 2.0 ** -8) - bound
        assert torch.equal(dx[past].double(), ref[past].sign() * float("inf"))
        worst = R.outside(dx[held], ref[held], bound[held])
        assert worst <= 1, worst
        assert bool(((dw.double() - wref).abs() <= wbound + R.U * wref.abs()).all())


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_fused_store(size, eps):
    """The very codes and scales of the 64-bit keys, and the separate call's q."""
    say("qk_norm_rope_store", size, eps)
    c = case(size)
    after = cache(c.t, c.hk, c.d)
    slots = torch.arange(c.t, dtype=torch.int32, device="cuda")
    q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how, eps=eps)
    assert torch.equal(q, F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how, eps=eps)[0])
    filled, empty = substitute(c.k, eps)
    codes, scale, sure, sure_scale = R.stored_turned(filled, c.kw, c.positions, c.freq, c.axes, eps, c.how["interleaved"])
    codes, scale = torch.where(empty, 0.0, codes), torch.where(empty[..., 0], 1.0, scale)
    assert float(sure.double().mean()) > 0.99
    assert bool(((R.values(after[0]) == codes) | ~sure).all())
    assert bool(((after[2] == scale) | ~sure_scale).all())


@pytest.mark.parametrize("power", [(120, 100), (-120, -100), (-133, 60), (127, -120)])
def test_fused_store_products_past_fp32(power):
    """Keys and weights whose product fp32 does not hold."""
    say("qk_norm_rope_store", power)
    c = Case(6, 2, 2, 64)
    c.k = torch.ldexp(c.k.double().clamp(-1, 1), torch.tensor(power[0], device="cuda")).to(BF)
    c.kw = torch.ldexp(c.kw.double(), torch.tensor(power[1], device="cuda")).to(BF)
    after = cache(c.t, c.hk, c.d)
    slots = torch.arange(c.t, dtype=torch.int32, device="cuda")
    F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how, eps=0.0)
    codes, scale, sure, sure_scale = c.stored_turned(0.0)
    assert float(sure.double().mean()) > 0.99
    assert bool(((R.values(after[0]) == codes) | ~sure).all())
    assert bool(((after[2] == scale) | ~sure_scale).all())


def test_other_heads_keep_their_bits():
    """A head's result does not depend on what the heads beside it are."""
    c = Case(40, 12, 4, 64, None, 3, False)
    ref = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)
    back = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    q, k = c.q.clone(), c.k.clone()
    q[::3, 1::4], k[1::5, 2], q[5, 5] = 0, 2.0 ** 90, 2.0 ** -130
    other = torch.ones(40, 12, dtype=torch.bool, device="cuda"), torch.ones(40, 4, dtype=torch.bool, device="cuda")
    other[0][::3, 1::4], other[1][1::5, 2], other[0][5, 5] = False, False, False
    for eps in (1e-6, 1e-20):
        base = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how, eps=eps) if eps != 1e-6 else ref
        grads = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how, eps=eps) if eps != 1e-6 else back
        got = F.fp8_qk_norm_rope(q, k, *c.table, **c.how, eps=eps)
        dgot = F.fp8_qk_norm_rope_backward(c.dq, c.dk, q, k, *c.table, **c.how, eps=eps)
        for i in range(2):
            assert torch.equal(got[i][other[i]], base[i][other[i]]) and torch.equal(dgot[i][other[i]], grads[i][other[i]])
