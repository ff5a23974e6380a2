"""The whole-number angles that the GPU tests of far positions compare with."""

from __future__ import annotations

import math
import random

import pytest

torch = pytest.importorskip("torch")

import qkv_angles as A  # noqa: E402
import qkv_ref as R  # noqa: E402


def angle(position, freq):
    q, r = A.rest(position, freq)
    assert abs(r) <= math.pi / 4 + 1e-15
    return complex(math.cos(r), math.sin(r)) * (1, 1j, -1, -1j)[q]


def fp32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def test_near_positions_against_fp64():
    """Below 2^-10 radians nothing is taken off and fp64's product is off by half a
    step alone; up to 2^10 its sine and cosine are good to 2^-53 of the angle."""
    rng = random.Random(1)
    for _ in range(2000):
        p, f = rng.randint(-1000, 1000), fp32(rng.random())
        want = complex(math.cos(p * f), math.sin(p * f))
        assert abs(angle(p, f) - want) <= 2.0 ** -52 * (1 + abs(p * f))


def test_far_positions_by_the_doubled_angle():
    """e^(i theta) at 2 p is its square at p, from 1 up to 2^31: a reduction that lost
    2^-51 of the angle would be off by 4e-7 at the far end."""
    rng = random.Random(2)
    for _ in range(300):
        f = fp32(rng.choice((1.0, rng.random(), 10.0 ** -rng.randint(1, 6))))
        p = rng.randint(1, 3)
        while 2 * p < 2 ** 31:
            z = angle(p, f)
            assert abs(angle(2 * p, f) - z * z) <= 2.0 ** -50
            p = 2 * p
    q, r = A.rest(2 ** 31 - 1, 1.0)
    z = angle(2 ** 31 - 1, 1.0) * angle(1, 1.0)
    assert abs(z - angle(2 ** 31, 1.0)) <= 2.0 ** -50 and abs(angle(-5, 0.75) * angle(5, 0.75) - 1) <= 2.0 ** -50


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn(interleaved):
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(5, 3, 32, generator=gen, dtype=torch.float64)
    positions = torch.randint(-50, 1000, (3, 5), generator=gen, dtype=torch.int32)
    freq = (100.0 ** (-torch.arange(8, dtype=torch.float64) / 8)).float()
    axes = tuple(i % 3 for i in range(8))
    cos, sin = A.turns(positions, freq, axes)
    want = R.turn(x, R.angles(positions, freq, axes), interleaved)
    assert float((A.turn(x, cos, sin, interleaved) - want).abs().max()) <= 2.0 ** -40
