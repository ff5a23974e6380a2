"""The 8-bit integer linear's tiles and K splits cover every accepted size, up to
rows next to 2^31, in numbers that its kernels hold."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
def test_cuts_cover_every_size(tmp_path):
    exe = str(tmp_path / "int8_cuts")
    subprocess.run([CXX, "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-ftrapv", "-I",
                    os.path.join(ROOT, "block_scaled_fp8_linear_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "int8_cuts.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout) > 4000
