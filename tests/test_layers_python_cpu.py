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


def calls(grad):
    """Each function on host tensors, with one input after another asking for
    a gradient."""
    t = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)  # noqa: E731
    x, y, b = t(2, 32), t(2, 24), t(24)
    q, s = torch.zeros(24, 32, dtype=torch.uint8), torch.zeros(1, 1)
    ask = lambda v: v.clone().requires_grad_(grad)  # noqa: E731
    yield lambda: F.fp8_block_linear_act(ask(x), q, s)
    yield lambda: F.fp8_block_linear_act(x, q, s, bias=ask(b))
    yield lambda: F.fp8_block_linear_act(x, q, s, residual=ask(y))
    yield lambda: F.fp8_block_linear_act_backward(ask(y), q, s)
    yield lambda: F.fp8_block_linear_act_backward(y, q, s, z=ask(y), act=F.ACT_SILU)
    yield lambda: F.fp8_block_glu(ask(x), q, s, q, s)
    yield lambda: F.fp8_block_glu_backward(ask(y), y, y, q, s, q, s)
    yield lambda: F.fp8_block_glu_backward(y, ask(y), y, q, s, q, s)
    yield lambda: F.fp8_block_glu_backward(y, y, ask(y), q, s, q, s)


def test_a_gradient_is_not_lost_in_silence():
    """While gradients are enabled an input that requires one is refused; under
    no_grad, and where none does, the call goes on (here to the refusal of
    host tensors)."""
    for call in calls(True):
        with pytest.raises(RuntimeError, match="not recorded by autograd"):
            call()
        with torch.no_grad(), pytest.raises(TypeError, match="device tensor"):
            call()
        with torch.inference_mode(), pytest.raises(TypeError, match="device tensor"):
            call()
    for call in calls(False):
        with pytest.raises(TypeError, match="device tensor"):
            call()
