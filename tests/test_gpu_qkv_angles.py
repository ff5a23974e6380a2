"""Rotation by far positions: the fused store's keys and scales are those of the exact
angle at every int32 position (tests/qkv_angles.py), not only where fp64's product of
position and frequency is exact.

The keys are computed in fp64: 2^-40 for the sine and cosine, and the norm's and the
turn's own roundings, at most (D + 40) 2^-53, so 2^-39 of |a| + |b| in all."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import qkv_angles as A  # noqa: E402
import qkv_ref as R  # noqa: E402
from test_gpu_qkv import Case, cache  # noqa: E402

OFF = 2.0 ** -39


def expected(c):
    """(keys, how far off they may be), both fp64."""
    x = c.k.double()
    n = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * c.kw.double()
    cos, sin = A.turns(c.positions, c.freq, c.axes)
    size, _ = R.reach(n, cos, c.how["interleaved"])
    return A.turn(n, cos, sin, c.how["interleaved"]), OFF * size


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [3000, 200000, 2 ** 24, 2 ** 31 - 1])
def test_keys_of_far_positions(far, interleaved):
    say("qk_norm_rope_store at", far)
    c = Case(50, 2, 6, 64, None, 3, interleaved, far=far)
    c.freq[0], c.freq[1] = 1.0, 0.9999
    c.positions[0, 0], c.positions[1, 1], c.positions[2, 2] = far, -far, 0
    if far > 2 ** 30:
        c.positions[1, 3] = -2 ** 31
    after = cache(50, 6, 64)
    slots = torch.arange(50, dtype=torch.int32, device="cuda")
    q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how)
    ref, off = expected(c)
    top, most, scale = ref.abs().amax(-1), off.amax(-1), R.scales(ref)
    sure = ((top - most) / 448.0).to(torch.float32) == ((top + most) / 448.0).to(torch.float32)

    def code(z):
        return R.nearest((z / scale.double()[..., None]).to(torch.float32).double())

    sure_code = sure[..., None] & (code(ref - off) == code(ref + off))
    assert float(sure.double().mean()) > 0.99 and float(sure_code.double().mean()) > 0.99
    wrong = int(((after[2] != scale) & sure).sum())
    assert wrong == 0, f"{wrong} of {scale.numel()} scales"
    assert bool(((R.values(after[0]) == code(ref)) | ~sure_code).all())
    assert torch.equal(q, F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)[0])


@pytest.mark.parametrize("freq", [2.0 ** 9, 2.0 ** 24, 1e30])
def test_frequencies_above_one(freq):
    """Angles to 2^40 exactly; any angle turns and does not stretch."""
    c = Case(30, 1, 4, 64, None, 1, True, far=2 ** 31 - 1)
    c.freq.fill_(freq)
    after = cache(30, 4, 64)
    slots = torch.arange(30, dtype=torch.int32, device="cuda")
    F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how)
    if freq == 2.0 ** 9:
        ref, off = expected(c)
        top, most, scale = ref.abs().amax(-1), off.amax(-1), R.scales(ref)
        sure = ((top - most) / 448.0).to(torch.float32) == ((top + most) / 448.0).to(torch.float32)
        assert bool(((after[2] == scale) | ~sure).all()) and float(sure.double().mean()) > 0.99
    keys = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)[1].double()
    x = c.k.double()
    n = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * c.kw.double()
    length = n[..., 0::2].square() + n[..., 1::2].square()
    got = keys[..., 0::2].square() + keys[..., 1::2].square()
    assert bool(((got - length).abs() <= 2.0 ** -6 * length + 1e-30).all())
