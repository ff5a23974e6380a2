"""Waits of the 8-bit integer kernels that stream the weight through LDS, read
from the assembly their source compiles to (tests/test_layers_isa_cpu.py has the
reading and its reason). Needs hipcc, no GPU."""

from __future__ import annotations

import os
import re
import subprocess

import pytest

from block_scaled_fp8_linear_amd import build as B
from test_layers_isa_cpu import _hipcc, outstanding_reads


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    if _hipcc() is None:
        pytest.skip("hipcc not available")

    def of(source):
        out = str(tmp_path_factory.mktemp("isa") / "listing.s")
        cmd = [_hipcc(), *B.COMMON_FLAGS, *B.FILE_FLAGS.get(source, []), "-I", B.INCLUDE, "-I", B.CSRC,
               "--cuda-device-only", "-S", os.path.join(B.CSRC, source), "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return open(out).read()

    return of


def test_slots_are_refilled_after_their_reads(listing):
    found = [f for f in outstanding_reads(listing("gemm_int8_skinny.hip")) if f[1] > 0]
    assert len(found) == 7, found
    assert not [f for f in found if f[2] > 0], found


def test_large_tiles_keep_the_products_fed(listing):
    """The 256 x 256 kernel: no spills, and no wait for loads among the products
    of a step but right ahead of its barrier (the compiler adds such waits where it can tell LDS arrays apart)."""
    text = listing("gemm_int8.hip")
    parts = [p for p in re.split(r"\n(?=_Z\w+:)", text) if "gemm_int8_kernelILi4ELi4ELi2ELb0E" in p.split(":")[0]]
    body = parts[0].split("s_endpgm")[0]
    assert "scratch_" not in body
    lines = [line.strip() for line in body.split("\n")]
    products = [i for i, line in enumerate(lines) if line.startswith("v_mfma_i32_32x32x32_i8")]
    assert products and len(products) % 64 == 0
    waits = 0
    for i in range(products[0], products[-1]):
        if lines[i].startswith("s_waitcnt") and "vmcnt" in lines[i]:
            behind = next(line for line in lines[i:] if line.startswith(("v_mfma", "s_barrier")))
            assert behind == "s_barrier", lines[i]
            waits += 1
    assert waits
