"""Every kernel form that the 8-bit integer linear's plans choose is run by a GPU
test: the plans (csrc/int8_plan.h) are compiled by themselves, asked over a wide grid
of sizes, and compared with the forms of the tested sizes."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

import int8_forms  # noqa: E402
import test_gpu_int8 as T  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
def test_every_form_is_tested(tmp_path):
    exe = str(tmp_path / "int8_forms")
    subprocess.run([CXX, "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "block_scaled_fp8_linear_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "int8_forms.cpp"), "-o", exe], check=True)
    scan = subprocess.run([exe, "scan"], capture_output=True, text=True, check=True).stdout.splitlines()
    reached = dict(line.split("\t") for line in scan)
    earlier = next(m for m in T.test_from_bf16.pytestmark if m.name == "parametrize").args[1]
    covered = [(*s, 0) for s in T.SHAPES + T.LARGE + int8_forms.CODES] + [(*s, 1) for s in earlier + int8_forms.FROM_BF16]
    lines = "\n".join(" ".join(map(str, t)) for t in covered)
    have = set(subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.splitlines())
    missing = {form: size for form, size in reached.items() if form not in have}
    assert len(reached) > 70 and not missing, missing
    for part in ("tiles of 256", "tiles of 128", "tiles of 64", "split", "several rounds", "whole lines", "odd rows", "K tail",
                 "one row, many columns, quantized on the way", "one row, few columns, quantized on the way", "two row tiles"):
        assert any(part in form for form in have), part
