"""Host-side checks of the layer operators' C ABI (include/fp8bl_layers.h):
exports, and argument errors as status codes before anything touches a
device. No pointer passed here is dereferenced."""

from __future__ import annotations

import pytest

from block_scaled_fp8_linear_amd import _lib as L

A = 1 << 24         # 16-byte aligned, far enough apart for the sizes below
OK, INVALID, ALIGN, WORK = L.FP8BL_OK, L.FP8BL_INVALID_ARG, L.FP8BL_ALIGNMENT, L.FP8BL_WORKSPACE
BIG_WS = (1 << 60, 1 << 50)


def test_exports():
    names = L.header_functions(L.LAYERS_HEADER_PATH)
    assert sorted(names) == sorted(f"fp8_block_{op}{end}" for op in
                                   ("linear_act", "linear_act_backward", "glu", "glu_backward")
                                   for end in ("", "_workspace_size"))
    for name in names:
        assert hasattr(L.load(), name)


@pytest.mark.parametrize("op", ["linear_act", "linear_act_backward", "glu", "glu_backward"])
def test_workspace_sizes(op):
    for m, n, k in [(0, 8, 16), (4, 0, 16), (4, 8, 15), (-1, 8, 16), (4, -8, 16), (4, 8, 0),
                    (4, (1 << 20) + 1, 16), (4, 8, (1 << 20) + 16), (1 << 31, 8, 16), (1 << 62, 1 << 62, 1 << 62)]:
        assert L.layer_workspace_size(op, m, n, k) == 0, (m, n, k)
    for m, n, k in [(1, 8000, 8192), (16, 5120, 5120), (512, 5120, 25600), (77, 1003, 656), (1, 1, 16)]:
        assert L.layer_workspace_size(op, m, n, k) % 256 == 0


SIZES = [
    (4, 8, 15, INVALID), (4, 8, 0, INVALID), (-1, 8, 16, INVALID), (4, -8, 16, INVALID),
    (1 << 31, 8, 16, INVALID), (4, (1 << 20) + 1, 16, INVALID), (4, 8, (1 << 20) + 16, INVALID),
    (1 << 20, 16, 1 << 16, INVALID), (1 << 20, 1 << 16, 16, INVALID), (0, 0, 16, OK),
]


@pytest.mark.parametrize("m,n,k,status", SIZES)
def test_size_errors(m, n, k, status):
    p = [(i + 1) << 40 for i in range(10)]
    assert L.linear_act_raw(*p[:7], m, n, k, 2, *BIG_WS) == status
    assert L.linear_act_backward_raw(*p[:7], m, n, k, 2, *BIG_WS) == status
    assert L.glu_raw(*p[:8], m, n, k, 2, *BIG_WS) == status
    assert L.glu_backward_raw(*p[:10], m, n, k, 2, *BIG_WS) == status


@pytest.mark.parametrize("act", [-1, 5, 99])
def test_unknown_activation(act):
    p = [(i + 1) * A for i in range(10)]
    assert L.linear_act_raw(*p[:7], 4, 8, 16, act, *BIG_WS) == INVALID
    assert L.linear_act_backward_raw(*p[:7], 4, 8, 16, act, *BIG_WS) == INVALID
    assert L.glu_raw(*p[:8], 4, 8, 16, act, *BIG_WS) == INVALID
    assert L.glu_backward_raw(*p[:10], 4, 8, 16, act, *BIG_WS) == INVALID


def _each(raw, count, optional, scales, size, act):
    """Every pointer in turn null, misaligned, and every pair overlapping."""
    base = [(i + 1) * A for i in range(count)]
    for i in range(count):
        if i not in optional:
            p = list(base)
            p[i] = 0
            assert raw(*p, *size, act, *BIG_WS) == INVALID, ("null", i)
        p = list(base)
        p[i] += 2 if i in scales else 8
        assert raw(*p, *size, act, *BIG_WS) == ALIGN, ("misaligned", i)
    return base


def test_linear_act_pointers():
    # x, q, s, bias, residual, z, y
    base = _each(L.linear_act_raw, 7, (3, 4, 5), (2,), (4, 24, 32), 2)
    for out in (5, 6):
        for other in range(7):
            if other == out or {out, other} == {4, 6}:
                continue
            p = list(base)
            p[out] = p[other]
            assert L.linear_act_raw(*p, 4, 24, 32, 2, *BIG_WS) == INVALID, (out, other)
    p = list(base)
    p[4] = p[6] + 48                  # residual overlaps y without being y
    assert L.linear_act_raw(*p, 4, 24, 32, 2, *BIG_WS) == INVALID
    assert L.linear_act_raw(*base, 0, 24, 32, 2, 0, 0) == OK
    assert L.linear_act_raw(0, 0, 0, 0, 0, 0, 0, 4, 0, 32, 2, 0, 0) == OK


def test_linear_act_backward_pointers():
    # dy, z, q, s, dz, dbias, dx
    base = _each(L.linear_act_backward_raw, 7, (5, 6), (3, 5), (4, 24, 32), 2)
    for out in (4, 5, 6):
        for other in range(7):
            if other == out:
                continue
            p = list(base)
            p[out] = p[other]
            assert L.linear_act_backward_raw(*p, 4, 24, 32, 2, *BIG_WS) == INVALID, (out, other)
    # without an activation there is neither z nor dz
    assert L.linear_act_backward_raw(*base, 4, 24, 32, 0, *BIG_WS) == INVALID
    assert L.linear_act_backward_raw(A, 0, 2 * A, 3 * A, 4 * A, 0, 5 * A, 4, 24, 32, 0, *BIG_WS) == INVALID
    # empty sums are written: their outputs are needed
    assert L.linear_act_backward_raw(0, 0, 0, 0, 0, 0, 0, 0, 24, 32, 0, 0, 0) == OK
    assert L.linear_act_backward_raw(0, 0, 0, 0, 0, 2, 0, 0, 24, 32, 0, 0, 0) == ALIGN
    assert L.linear_act_backward_raw(0, 0, 0, 0, 0, 0, 8, 4, 0, 32, 0, 0, 0) == ALIGN


def test_glu_pointers():
    # x, qg, sg, qu, su, g, u, h
    base = _each(L.glu_raw, 8, (5, 6), (2, 4), (4, 24, 32), 2)
    for out in (5, 6, 7):
        for other in range(8):
            if other == out:
                continue
            p = list(base)
            p[out] = p[other]
            assert L.glu_raw(*p, 4, 24, 32, 2, *BIG_WS) == INVALID, (out, other)
    for lone in (5, 6):               # g and u go together
        p = list(base)
        p[lone] = 0
        assert L.glu_raw(*p, 4, 24, 32, 2, *BIG_WS) == INVALID


def test_glu_backward_pointers():
    # dh, g, u, qg, sg, qu, su, dg, du, dx
    base = _each(L.glu_backward_raw, 10, (9,), (4, 6), (4, 24, 32), 2)
    for out in (7, 8, 9):
        for other in range(10):
            if other == out:
                continue
            p = list(base)
            p[out] = p[other]
            assert L.glu_backward_raw(*p, 4, 24, 32, 2, *BIG_WS) == INVALID, (out, other)


@pytest.mark.parametrize("op,raw,pointers", [
    ("linear_act", L.linear_act_raw, 7), ("linear_act_backward", L.linear_act_backward_raw, 7),
    ("glu", L.glu_raw, 8), ("glu_backward", L.glu_backward_raw, 10)])
def test_workspace_errors(op, raw, pointers):
    """At a size that needs one: missing, short, misaligned, over an input."""
    shape = next((t for t in [(16, 4003, 8192), (300, 1003, 25600)] if L.layer_workspace_size(op, *t) > 0), None)
    if shape is None:
        pytest.skip("needs no workspace at these sizes")
    need = L.layer_workspace_size(op, *shape)
    p = [(i + 1) << 40 for i in range(pointers)]
    assert raw(*p, *shape, 2, 0, 0) == WORK
    assert raw(*p, *shape, 2, 1 << 50, need - 1) == WORK
    assert raw(*p, *shape, 2, (1 << 50) + 128, need) == ALIGN
    assert raw(*p, *shape, 2, p[0], need) == INVALID
