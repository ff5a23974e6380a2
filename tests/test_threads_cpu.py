"""Calls of the compiled functions from several threads, as far as they go without a
device, and the helper that the GPU test of threads rests on."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import block_scaled_fp8_linear_amd as F  # noqa: E402
from threads import together  # noqa: E402


def test_a_thread_that_raises_is_reported():
    assert together(lambda: 1, lambda: 2) == [1, 2]
    with pytest.raises(AssertionError, match="thread 1 raised ValueError: no"):
        together(lambda: 1, lambda: exec("raise ValueError('no')"))


def test_refusals_in_two_threads():
    i8, f = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)

    def work():
        for _ in range(300):
            with pytest.raises(TypeError, match="device tensor"):
                F.int8_linear(i8, f, i8, f)
            with pytest.raises(TypeError, match="missing argument 'slots'"):
                F.fp8_kv_store(i8, i8)
        return True

    assert together(work, work, work) == [True] * 3
