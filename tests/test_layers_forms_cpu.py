"""Every kernel form that the layer operators' plans choose is run by a GPU
test: the plans (csrc/layer_plan.h) are compiled by themselves, asked over a
wide grid of sizes, and compared with the forms of the tested sizes."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

import layers_forms  # noqa: E402
import test_gpu_layers as T  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
OPS = ("linear_act", "linear_act_backward", "glu", "glu_backward")


def covered():
    for op in OPS:
        for shape in T.SHAPES + T.LARGE + layers_forms.FORMS[op]:
            yield (op, *shape)
    yield "linear_act_backward", 2048, 4096, 8448       # test_large_columns_left_over
    yield "linear_act", 2048, 8448, 4096


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
def test_every_form_is_tested(tmp_path):
    exe = str(tmp_path / "layer_forms")
    subprocess.run([CXX, "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "block_scaled_fp8_linear_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "layer_forms.cpp"), "-o", exe], check=True)
    scan = subprocess.run([exe, "scan"], capture_output=True, text=True, check=True).stdout.splitlines()
    reached = dict(line.split("\t") for line in scan)
    lines = "\n".join(" ".join(map(str, t)) for t in covered())
    have = set(subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.splitlines())
    missing = {form: size for form, size in reached.items() if form not in have}
    assert len(reached) > 100 and not missing, missing
    # each tile and both of its ends, each stream
    for part in ("256-row", "128-row", "64-row", "split", "unsplit", "odd rows", "few rows", "whole rounds",
                 "columns left over", "join of quads", "X in LDS", "X in registers"):
        assert any(part in form for form in have), part
