"""What the layer operators' Python functions take and refuse, as far as no
device is needed."""

from __future__ import annotations

import inspect

import pytest

torch = pytest.importorskip("torch")

import block_scaled_fp8_linear_amd as F  # noqa: E402


@pytest.mark.parametrize("name", ["fp8_block_linear_act_backward", "fp8_block_glu_backward"])
def test_the_input_gradient_can_be_left_out(name):
    assert inspect.signature(getattr(F, name)).parameters["need_dx"].default is True
