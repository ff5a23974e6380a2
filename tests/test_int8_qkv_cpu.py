"""Host-side checks of include/fp8bl_int8.h and include/fp8bl_qkv.h: exports,
the argument structure, and argument errors as status codes before anything
touches a device. No pointer passed here is dereferenced but the structure's."""

from __future__ import annotations

import re

import pytest

torch = pytest.importorskip("torch")

import block_scaled_fp8_linear_amd as F  # noqa: E402
from block_scaled_fp8_linear_amd import _lib as L  # noqa: E402

OK, INVALID, ALIGN, WORK = L.FP8BL_OK, L.FP8BL_INVALID_ARG, L.FP8BL_ALIGNMENT, L.FP8BL_WORKSPACE
A = 1 << 32
BIG = (1 << 60, 1 << 50)


def test_exports():
    assert set(L.header_functions(L.INT8_HEADER_PATH)) == {
        "int8_row_quantize", "int8_row_quantize_bf16", "int8_linear", "int8_linear_workspace_size", "int8_linear_bf16",
        "int8_linear_bf16_workspace_size"}
    assert set(L.header_functions(L.QKV_HEADER_PATH)) == {
        "fp8_qk_norm_rope", "fp8_qk_norm_rope_backward", "fp8_qk_norm_rope_backward_workspace_size", "fp8_kv_store",
        "fp8_kv_load", "fp8_qk_norm_rope_store"}
    for path in (L.INT8_HEADER_PATH, L.QKV_HEADER_PATH):
        for name in L.header_functions(path):
            assert hasattr(L.load(), name)
    for name in ("int8_row_quantize", "int8_linear", "int8_linear_bf16", "fp8_qk_norm_rope", "fp8_qk_norm_rope_backward",
                 "fp8_kv_store", "fp8_kv_load", "fp8_qk_norm_rope_store"):
        assert name in F.__all__ and getattr(F, name).__doc__


def test_structure_follows_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(L.QKV_HEADER_PATH).read(), flags=re.S)
    body = re.search(r"typedef struct fp8bl_qkv \{(.*?)\} fp8bl_qkv;", text, re.S).group(1)
    members = []
    for line in body.split(";"):
        words = line.replace("*", " ").split()
        if not words:
            continue
        names = [n.strip() for n in " ".join(words).split(",")]
        names[0] = names[0].split()[-1]
        for n in names:
            if "fp8bl_heads" in words:
                members += [f"{n}_data", f"{n}_token_stride", f"{n}_head_stride"]
            elif "[" not in n:
                members.append(n)
    assert tuple(members) == L._QKV_FIELDS
    assert re.search(r"define FP8BL_MAX_PAIRS (\d+)", text).group(1) == str(L.MAX_PAIRS)
    assert re.search(r"define FP8BL_MAX_AXES (\d+)", text).group(1) == str(L.MAX_AXES)
    assert len(L.qkv_struct()) == 8 * len(L._QKV_FIELDS) + L.MAX_PAIRS


# ---- 8-bit integer linear ----------------------------------------------

@pytest.mark.parametrize("m,n,k,status", [
    (4, 8, 15, INVALID), (4, 8, 0, INVALID), (4, 8, -16, INVALID), (-1, 8, 16, INVALID), (4, -8, 16, INVALID),
    (1 << 31, 8, 16, INVALID), (4, (1 << 20) + 1, 16, INVALID), (4, 8, 1 << 17, INVALID), (1 << 30, 64, 16, INVALID),
    (1 << 30, 8, 64, INVALID), (1 << 62, 1 << 62, 1 << 62, INVALID), (0, 0, 16, OK), (0, 8, 16, OK), (4, 0, 16, OK)])
def test_int8_sizes(m, n, k, status):
    p = [(i + 1) << 44 for i in range(6)]
    assert L.int8_linear_raw(*p, m, n, k, *BIG) == status
    assert L.int8_linear_bf16_raw(*p[:5], m, n, k, *BIG) == status
    if n == 8:
        for bf16 in (False, True):
            assert L.int8_row_quantize_raw(*p[:3], m, k, bf16) == status
    if status == INVALID or m * n == 0:
        assert L.int8_workspace_size(m, n, k) == 0 and L.int8_workspace_size(m, n, k, False) == 0


def test_int8_pointers():
    p = [(i + 1) * A for i in range(6)]         # xq, xs, wq, ws, bias, y
    size = (4, 24, 32)
    for i in range(6):
        bad = list(p)
        bad[i] += 2 if i in (1, 3) else 8
        assert L.int8_linear_raw(*bad, *size, *BIG) == ALIGN
        if i != 4:
            bad[i] = 0
            assert L.int8_linear_raw(*bad, *size, *BIG) == INVALID
        if i != 5:
            bad = list(p)
            bad[5] = p[i]
            assert L.int8_linear_raw(*bad, *size, *BIG) == INVALID
    p = [p[0], *p[2:]]                          # x, wq, ws, bias, y
    for i in range(5):
        bad = list(p)
        bad[i] += 2 if i == 2 else 8
        assert L.int8_linear_bf16_raw(*bad, *size, *BIG) == ALIGN
        if i != 3:
            bad[i] = 0
            assert L.int8_linear_bf16_raw(*bad, *size, *BIG) == INVALID
        if i != 4:
            bad = list(p)
            bad[4] = p[i]
            assert L.int8_linear_bf16_raw(*bad, *size, *BIG) == INVALID
    for bf16 in (False, True):
        assert L.int8_row_quantize_raw(0, A, 2 * A, 4, 32, bf16) == INVALID
        assert L.int8_row_quantize_raw(A, 0, 2 * A, 4, 32, bf16) == INVALID
        assert L.int8_row_quantize_raw(A, 2 * A, 0, 4, 32, bf16) == INVALID
        assert L.int8_row_quantize_raw(A + 8, 2 * A, 3 * A, 4, 32, bf16) == ALIGN
        assert L.int8_row_quantize_raw(A, 2 * A + 8, 3 * A, 4, 32, bf16) == ALIGN
        assert L.int8_row_quantize_raw(A, 2 * A, 3 * A + 2, 4, 32, bf16) == ALIGN
        assert L.int8_row_quantize_raw(A, A + 64, 3 * A, 4, 32, bf16) == INVALID
        assert L.int8_row_quantize_raw(A, 2 * A, 2 * A + 64, 4, 32, bf16) == INVALID


@pytest.mark.parametrize("shape", [(1, 8000, 8192), (16, 5120, 5120), (333, 4300, 1168), (512, 5120, 25600), (8192, 12288, 4096),
                                   (1, 1, 16)])
def test_int8_workspace(shape):
    p = [(i + 1) << 44 for i in range(5)]
    need = L.int8_workspace_size(*shape)
    assert need % 256 == 0 and need >= shape[0] * shape[2] + 4 * shape[0]
    assert L.int8_linear_bf16_raw(*p, *shape, 0, 0) == WORK
    assert L.int8_linear_bf16_raw(*p, *shape, 1 << 50, need - 1) == WORK
    assert L.int8_linear_bf16_raw(*p, *shape, (1 << 50) + 128, need) == ALIGN
    assert L.int8_linear_bf16_raw(*p, *shape, p[0], need) == INVALID


# ---- from the QKV projection to its cache -------------------------------

T, HQ, HK, D = 4, 6, 2, 32
BASE = {"tokens": T, "q_heads": HQ, "k_heads": HK, "head_dim": D, "axes": 2, "pairs": 16, "interleaved": 0, "eps": 1e-6,
        "cache_rows": 10}
HEADS = {"q": HQ, "k": HK, "v": HK, "q_out": HQ, "k_out": HK, "v_out": HK, "dq": HQ, "dk": HK}
for _i, (_name, _h) in enumerate(HEADS.items()):
    BASE |= {f"{_name}_data": (_i + 1) * A, f"{_name}_token_stride": _h * D, f"{_name}_head_stride": D}
PLAIN = ("q_weight", "k_weight", "dq_weight", "dk_weight", "positions", "inv_freq", "slots", "k_cache", "v_cache", "k_scale",
         "v_scale")
BASE |= {name: (20 + i) * A for i, name in enumerate(PLAIN)}
AXIS = bytes([0, 1] * 8)

CALLS = {
    "rope": (L.qk_norm_rope_raw, ("q", "k"), ("q_out", "k_out"), ("q_weight", "k_weight", "positions", "inv_freq"), ()),
    "back": (lambda s: L.qk_norm_rope_backward_raw(s, *BIG), ("q", "k", "dq", "dk"), ("q_out", "k_out"),
             ("q_weight", "k_weight", "positions", "inv_freq"), ("dq_weight", "dk_weight")),
    "store": (L.kv_store_raw, ("k", "v"), (), ("slots",), ("k_cache", "v_cache", "k_scale", "v_scale")),
    "load": (L.kv_load_raw, (), ("k_out", "v_out"), ("slots", "k_cache", "v_cache", "k_scale", "v_scale"), ()),
    "fused": (L.qk_norm_rope_store_raw, ("q", "k", "v"), ("q_out",),
              ("q_weight", "k_weight", "positions", "inv_freq", "slots"), ("k_cache", "v_cache", "k_scale", "v_scale")),
}
TURNS, CACHES = ("rope", "back", "fused"), ("store", "load", "fused")


def status(call, axis=AXIS, **changed):
    return CALLS[call][0](L.qkv_struct(axis, **(BASE | changed)))


@pytest.mark.parametrize("call", CALLS)
def test_qkv_sizes(call):
    for changed in ({"tokens": -1}, {"tokens": 1 << 31}, {"k_heads": -1}, {"k_heads": 4097}, {"head_dim": 8},
                    {"head_dim": 36}, {"head_dim": 264}, {"head_dim": 0}, {"head_dim": -16}, {"tokens": 1 << 62}):
        assert status(call, **changed) == INVALID, changed
    if call in TURNS:
        for changed in ({"q_heads": -1}, {"q_heads": 4097}, {"axes": 0}, {"axes": 9}, {"axes": 1}, {"pairs": 0},
                        {"pairs": 12}, {"pairs": 24}, {"pairs": -8}, {"pairs": 136}, {"pairs": 6, "interleaved": 1},
                        {"interleaved": 2}, {"interleaved": -1}, {"eps": -1e-6}, {"eps": float("nan")},
                        {"eps": float("inf")}, {"eps": 1e300}, {"axis": bytes([0, 2] * 8)}, {"axis": bytes([255] * 16)}):
            assert status(call, **changed) == INVALID, changed
    if call in CACHES:
        for changed in ({"cache_rows": -1}, {"cache_rows": 1 << 31}):
            assert status(call, **changed) == INVALID, changed
    if call in ("store", "fused"):
        assert status(call, tokens=65537) == INVALID
    assert CALLS[call][0](None) == INVALID
    assert status(call, tokens=0, **{name: 0 for name in PLAIN}) == OK


@pytest.mark.parametrize("call", CALLS)
def test_qkv_pointers(call):
    _, heads_in, heads_out, plain_in, plain_out = CALLS[call]
    everything = [f"{h}_data" for h in heads_in + heads_out] + list(plain_in + plain_out)
    four = ("positions", "inv_freq", "slots", "k_scale", "v_scale", "dq_weight", "dk_weight")
    for name in everything:
        if name not in ("dq_weight", "dk_weight"):
            assert status(call, **{name: 0}) == INVALID, name
        assert status(call, **{name: BASE[name] + (2 if name in four else 8)}) == ALIGN, name
    for out in [f"{h}_data" for h in heads_out] + list(plain_out):
        for other in everything:
            if other == out or {out, other} in ({"q_data", "q_out_data"}, {"k_data", "k_out_data"}):
                if call != "back" or other == out:
                    continue
            if call == "back" and {out, other} in ({"dq_data", "q_out_data"}, {"dk_data", "k_out_data"}):
                continue
            assert status(call, **{out: BASE[other]}) == INVALID, (out, other)


@pytest.mark.parametrize("call", CALLS)
def test_qkv_strides(call):
    _, heads_in, heads_out, _, _ = CALLS[call]
    for h in heads_in + heads_out:
        for part in ("token", "head"):
            for bad in (-8, 12, 1 << 41, -(1 << 62), 1 << 62):
                assert status(call, **{f"{h}_{part}_stride": bad}) == INVALID, (h, part, bad)
    for h in heads_out:                       # elements that coincide
        assert status(call, **{f"{h}_token_stride": 0}) == INVALID
        assert status(call, **{f"{h}_head_stride": 0}) == INVALID
        assert status(call, **{f"{h}_head_stride": D - 8}) == INVALID
        assert status(call, **{f"{h}_token_stride": HEADS[h] * D - 8}) == INVALID
        assert status(call, **{f"{h}_token_stride": D, f"{h}_head_stride": T * D - 8}) == INVALID


def _gated(st):
    """Past every check: no device here, or one that is not asked."""
    return st in (L.FP8BL_HIP_ERROR, L.FP8BL_UNSUPPORTED_DEVICE)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers would reach the device")
def test_what_is_taken():
    for call in CALLS:
        assert _gated(status(call)), call
    row = (HQ + 2 * HK) * D
    at = {"q": 0, "k": HQ * D * 2, "v": (HQ + HK) * D * 2}
    packed = {}
    for h, off in at.items():
        packed |= {f"{h}_data": A + off, f"{h}_token_stride": row}
    outs = {f"{h}_out_{part}": packed[f"{h}_{part}"] for h in ("q", "k") for part in ("data", "token_stride")}
    assert _gated(status("rope", **packed, **outs))                  # in place in one packed array
    assert _gated(status("fused", **packed, **{n: v for n, v in outs.items() if n.startswith("q")}))
    swapped = dict(outs, q_out_data=outs["k_out_data"], k_out_data=outs["q_out_data"] + row * 2 * T)
    assert status("rope", **packed, **swapped) == INVALID            # q over k
    shifted = dict(outs, q_out_data=outs["q_out_data"] + 16)
    assert status("rope", **packed, **shifted) == INVALID
    # the same array as q and as k, q in place: k would be read after it
    same = {"k_heads": HQ, "k_data": BASE["q_data"], "k_token_stride": HQ * D, "k_out_token_stride": HQ * D,
            "q_out_data": BASE["q_data"]}
    assert status("rope", **same) == INVALID
    grads = {f"{g}_{part}": BASE[f"{o}_{part}"] for g, o in (("q_out", "dq"), ("k_out", "dk")) for part in ("data",)}
    assert _gated(status("back", **grads))
    first = {"q_out_token_stride": D, "q_out_head_stride": T * D}
    assert _gated(status("rope", **first))
    assert _gated(status("rope", tokens=1, q_token_stride=3, q_out_token_stride=-5))      # no second token
    assert _gated(status("back", dq_weight=0, dk_weight=0))
    assert _gated(status("load", k_token_stride=3, eps=float("nan"), pairs=1 << 40, axes=-1, q_heads=-1))   # not read
    assert _gated(status("store", pairs=1 << 40, axes=-1, q_heads=1 << 50, eps=float("nan")))


def test_backward_workspace():
    size = F.qk_norm_rope_backward_workspace_size
    for bad in ((-1, 2, 2, 64), (4, -1, 2, 64), (4, 2, 2, 60), (1 << 62, 2, 2, 64), (0, 2, 2, 64), (4, 0, 0, 64)):
        assert size(*bad) == 0
    need = size(T, HQ, HK, D)
    assert need > 0 and need % 256 == 0 and size((1 << 31) - 1, 4096, 4096, 256) <= 1 << 22
    s = L.qkv_struct(AXIS, **BASE)
    assert L.qk_norm_rope_backward_raw(s, 0, 0) == WORK
    assert L.qk_norm_rope_backward_raw(s, 1 << 50, need - 1) == WORK
    assert L.qk_norm_rope_backward_raw(s, (1 << 50) + 128, need) == ALIGN
    assert L.qk_norm_rope_backward_raw(s, BASE["dq_data"], need) == INVALID


def test_tensor_arguments():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 32, dtype=torch.bfloat16)
    i8, f = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    pos, freq, w = torch.zeros(2, dtype=torch.int32), torch.zeros(16), torch.zeros(32, dtype=torch.bfloat16)
    codes, scale = torch.zeros(3, 4, 32, dtype=torch.uint8), torch.zeros(3, 4)
    slots = torch.zeros(2, dtype=torch.int32)
    cache = (codes, codes, scale, scale)
    calls = [lambda: F.int8_row_quantize(x), lambda: F.int8_linear(i8, f, i8, f), lambda: F.int8_linear_bf16(x, i8, f),
             lambda: F.fp8_qk_norm_rope(q, q, w, w, pos, freq),
             lambda: F.fp8_qk_norm_rope_backward(q, q, q, q, w, w, pos, freq),
             lambda: F.fp8_kv_store(q, q, slots, *cache), lambda: F.fp8_kv_load(*cache, slots),
             lambda: F.fp8_qk_norm_rope_store(q, q, q, w, w, pos, freq, slots, *cache)]
    for call in calls:
        with pytest.raises(TypeError, match="device tensor"):
            call()
    x.requires_grad_(True)
    q.requires_grad_(True)
    for i in (0, 2, 3, 4, 5, 7):
        with pytest.raises(RuntimeError, match="autograd"):
            calls[i]()
        with torch.no_grad(), pytest.raises(TypeError, match="device tensor"):
            calls[i]()


def test_compiled_calls_check_their_parameters():
    i8, f = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    for call, text in ((lambda: F.int8_linear(i8, f, i8), "missing argument 'w_scale'"),
                       (lambda: F.int8_linear(i8, f, i8, f, None, None, None, 1), "at most 7"),
                       (lambda: F.int8_linear(i8, f, i8, f, scale=f), "unexpected keyword argument 'scale'"),
                       (lambda: F.int8_linear(i8, f, i8, f, xq=i8), "multiple values"),
                       (lambda: F.int8_linear(3, f, i8, f), "xq must be a tensor"),
                       (lambda: F.fp8_kv_store(k=i8, v=i8), "missing argument")):
        with pytest.raises(TypeError, match=text):
            call()
    with pytest.raises(AttributeError):
        F.no_such_function
    # keyword names that are not the interned ones
    with pytest.raises(TypeError, match="device tensor"):
        F.int8_linear(i8, f, **{"".join(["w", "q"]): i8, "".join(["w_", "scale"]): f})


def test_names_without_the_library(monkeypatch):
    """Not built: the compiled functions are there like the others, and raise when
    they are called."""
    for name in F._COMPILED:
        monkeypatch.delitem(vars(F), name, raising=False)
    monkeypatch.setattr(F._lib, "_lib", None)
    monkeypatch.setattr(F._lib, "LIB_PATH", "/nowhere/libfp8bl.so")
    for name in F._COMPILED:
        with pytest.raises(ImportError, match="not built"):
            getattr(F, name)()
    monkeypatch.undo()
    with pytest.raises(TypeError, match="missing argument"):
        F.int8_linear()
