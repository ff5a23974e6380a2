"""The compiled functions (binding/tensors.cpp) beside the rest of torch: tensors that
they write, and errors."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
from test_binding_autograd_cpu import NAMES, calls  # noqa: E402

BF = torch.bfloat16
WRITTEN = {"int8_row_quantize": ("q", "scale"), "int8_linear": ("out",), "int8_linear_bf16": ("out",),
           "fp8_qk_norm_rope": ("q_out", "k_out"), "fp8_qk_norm_rope_backward": ("q_grad", "k_grad"),
           "fp8_kv_store": ("k_cache", "v_cache", "k_scale", "v_scale"), "fp8_kv_load": ("k_out", "v_out"),
           "fp8_qk_norm_rope_store": ("k_cache", "v_cache", "k_scale", "v_scale", "q_out")}
OPTIONAL = ("out", "q_out", "k_out", "v_out", "q_grad", "k_grad")


def on_gpu(name):
    return {k: v.cuda() for k, v in calls()[name].items()}


@pytest.mark.parametrize("name", NAMES)
def test_versions_of_written_tensors(name):
    """Written tensors get a new version, the others and new outputs do not; views
    count with their base."""
    say("versions", name)
    args = on_gpu(name)
    before = {k: v._version for k, v in args.items()}
    getattr(F, name)(**args)
    assert {k for k, v in args.items() if v._version != before[k]} == set(WRITTEN[name])
    for param in WRITTEN[name]:
        args = on_gpu(name)
        base = torch.zeros(2, *args[param].shape, dtype=args[param].dtype, device="cuda")
        args[param] = base[0]
        version = base._version
        getattr(F, name)(**args)
        assert base._version > version
    args = {k: v for k, v in on_gpu(name).items() if k not in OPTIONAL + (("q", "scale") if name == "int8_row_quantize" else ())}
    got = getattr(F, name)(**args)
    for t in got if isinstance(got, tuple) else (got,):
        assert t is None or t._version == 0


@pytest.mark.parametrize("name", NAMES)
def test_inference_tensors(name):
    """They have no versions, and are taken as before."""
    with torch.inference_mode():
        args = on_gpu(name)
        getattr(F, name)(**args)
    getattr(F, name)(**args)


def test_a_saved_tensor_that_is_turned_in_place_is_noticed():
    args = on_gpu("fp8_qk_norm_rope")
    q = torch.randn(2, 4, 32, device="cuda").to(BF)
    weight = torch.ones(32, dtype=BF, device="cuda", requires_grad=True)
    loss = (q * weight).sum()                      # saves q
    with torch.no_grad():
        F.fp8_qk_norm_rope(**(args | {"q": q, "q_out": q}))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_out_of_memory_is_torchs_error():
    """2 TiB of keys and as many values: torch's own error, by which callers free and
    try again; the call after it works."""
    cache = [torch.zeros(1, 4096, 256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones(1, 4096, device="cuda") for _ in range(2)]
    slots = torch.zeros(1 << 20, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError, match="out of memory") as e:
        F.fp8_kv_load(*cache, slots)
    assert "frame #" not in str(e.value)
    k, v = F.fp8_kv_load(*cache, slots[:3])
    assert k.shape == v.shape == (3, 4096, 256)
