"""What the compiled functions (binding/tensors.cpp) refuse of autograd's tensors.
The refusals come before any look at devices, so CPU tensors show them."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import block_scaled_fp8_linear_amd as F  # noqa: E402

BF = torch.bfloat16


def calls():
    """name -> (function, arguments by name). Every tensor that may be given is."""
    x, q = torch.zeros(2, 32, dtype=BF), torch.zeros(2, 4, 32, dtype=BF)
    i8, f = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    table = {"q_weight": torch.zeros(32, dtype=BF), "k_weight": torch.zeros(32, dtype=BF),
             "positions": torch.zeros(2, dtype=torch.int32), "inv_freq": torch.zeros(16)}
    cache = {n: torch.zeros(3, 4, 32, dtype=torch.uint8) for n in ("k_cache", "v_cache")}
    cache |= {n: torch.zeros(3, 4) for n in ("k_scale", "v_scale")}
    slots = {"slots": torch.zeros(2, dtype=torch.int32)}

    def heads(*names):
        return {n: q.clone() for n in names}

    return {
        "int8_row_quantize": {"x": x.clone(), "q": i8.clone(), "scale": f.clone()},
        "int8_linear": {"xq": i8, "x_scale": f.clone(), "wq": i8, "w_scale": f.clone(), "bias": torch.zeros(2, dtype=BF),
                        "out": torch.zeros(2, 2, dtype=BF)},
        "int8_linear_bf16": {"x": x.clone(), "wq": i8, "w_scale": f.clone(), "bias": torch.zeros(2, dtype=BF),
                             "out": torch.zeros(2, 2, dtype=BF)},
        "fp8_qk_norm_rope": heads("q", "k") | table | heads("q_out", "k_out"),
        "fp8_qk_norm_rope_backward": heads("dq", "dk", "q", "k") | table | heads("q_grad", "k_grad"),
        "fp8_kv_store": heads("k", "v") | slots | cache,
        "fp8_kv_load": cache | slots | heads("k_out", "v_out"),
        "fp8_qk_norm_rope_store": heads("q", "k", "v") | table | slots | cache | heads("q_out"),
    }


NAMES = list(calls())
INPUT = {"int8_row_quantize": "x", "int8_linear": "w_scale", "int8_linear_bf16": "x", "fp8_qk_norm_rope": "q",
         "fp8_qk_norm_rope_backward": "dq", "fp8_kv_store": "k", "fp8_qk_norm_rope_store": "k"}


@pytest.mark.parametrize("name", INPUT)
def test_the_refusal_names_functions_that_exist(name):
    args = calls()[name]
    args[INPUT[name]].requires_grad_(True)
    with pytest.raises(RuntimeError, match="not recorded by autograd") as e:
        getattr(F, name)(**args)
    text = str(e.value)
    assert "torch.no_grad()" in text
    if name == "fp8_qk_norm_rope":
        assert "with fp8_qk_norm_rope_backward, or" in text
    else:
        assert "torch.autograd.Function" not in text and "there is no backward function" in text
    with torch.no_grad(), pytest.raises(TypeError, match="device tensor"):
        getattr(F, name)(**args)


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_that_requires_grad_is_refused(name):
    """Scales, frequencies and given outputs among them."""
    floats = [k for k, v in calls()[name].items() if v.is_floating_point()]
    assert floats
    for param in floats:
        args = calls()[name]
        args[param].requires_grad_(True)
        with pytest.raises(RuntimeError, match=f"autograd and {param} requires grad"):
            getattr(F, name)(**args)
        args[param] = args[param] * 2                    # not a leaf
        with pytest.raises(RuntimeError, match=f"autograd and {param} requires grad"):
            getattr(F, name)(**args)
        with torch.no_grad(), pytest.raises(TypeError, match="device tensor"):
            getattr(F, name)(**args)


@pytest.mark.parametrize("name", NAMES)
def test_a_tangent_is_refused(name):
    """Forward mode: a dual tensor's tangent would be lost, under no_grad too."""
    ad = torch.autograd.forward_ad
    for param in (k for k, v in calls()[name].items() if v.is_floating_point()):
        args = calls()[name]
        with ad.dual_level():
            args[param] = ad.make_dual(args[param], torch.ones_like(args[param]))
            with pytest.raises(RuntimeError, match=f"autograd and {param} has a tangent"):
                getattr(F, name)(**args)
            with torch.no_grad(), pytest.raises(RuntimeError, match=f"{param} has a tangent"):
                getattr(F, name)(**args)
            args[param] = ad.unpack_dual(args[param]).primal
            with pytest.raises(TypeError, match="device tensor"):
                getattr(F, name)(**args)
