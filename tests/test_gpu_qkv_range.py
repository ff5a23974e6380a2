"""Norm and rotation of heads whose values leave the range of fp32 on the way. The
definitions and bounds are those of tests/qkv_ref.py."""

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
