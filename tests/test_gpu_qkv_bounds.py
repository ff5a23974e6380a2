"""Norm, rotation and their gradients within bounds that leave no room for a coarser
angle (tests/qkv_bounds.py), at the sizes of tests/test_gpu_qkv.py, at ordinary and at
far positions."""

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
import qkv_bounds as B  # noqa: E402
import qkv_ref as R  # noqa: E402
from test_gpu_qkv import CASES, Case  # noqa: E402

FAR = [(size, 1000) for size in CASES] + [((60, 6, 2, 64, None, 3, inter), far) for inter in (False, True)
                                           for far in (200000, 2 ** 31 - 1)]
IDS = ["-".join(str(int(v)) if v is not None else "all" for v in size) + f"-to-{far}" for size, far in FAR]


@pytest.mark.parametrize("size,far", FAR, ids=IDS)
def test_norm_rope_and_gradients(size, far):
    say("qk_norm_rope", size, far)
    c = Case(*size, far=far)
    cos, sin = A.turns(c.positions, c.freq, c.axes)
    inter = c.how["interleaved"]
    q, k = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)
    for got, x, w in ((q, c.q, c.qw), (k, c.k, c.kw)):
        worst = R.outside(got, *B.forward(x, w, cos, sin, 1e-6, inter))
        assert worst <= 1, worst
    lanes = next(n for n in (2, 4, 8, 16, 32) if 8 * n >= c.d)
    back = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    for dx, dw, dy, x, w in ((back[0], back[2], c.dq, c.q, c.qw), (back[1], back[3], c.dk, c.k, c.kw)):
        steps = -(-x.shape[1] * lanes // 64) * -(-c.t // 4096)
        ref, bound, wref, wbound = B.backward(dy, x, w, cos, sin, 1e-6, inter, steps)
        worst = R.outside(dx, ref, bound)
        assert worst <= 1, worst
        assert bool(((dw.double() - wref).abs() <= wbound + B.U * wref.abs()).all())
