"""Waits of the streaming kernels, read from the assembly the library's own
sources compile to. Needs hipcc, no GPU.

In these kernels a wave refills the ring slot that it has just read, with loads
that write LDS on their own. A read that has been issued but has not returned
would then race with the refill, so every such load needs the wave's LDS reads
to have returned (lgkmcnt 0) before it is issued."""

from __future__ import annotations

import os
import re
import subprocess

import pytest

from block_scaled_fp8_linear_amd import build as B


def _hipcc():
    try:
        return B.hipcc()
    except RuntimeError:
        return None


def outstanding_reads(text):
    """(kernel, loads into LDS, the most LDS reads not waited for at one of
    them) for each kernel of an assembly listing, in its order."""
    found = []
    for part in re.split(r"\n(?=_Z\w+:)", text):
        name = part.split(":")[0]
        if not name.startswith("_Z"):
            continue
        reads = worst = loads = 0
        for line in part.split("s_endpgm")[0].split("\n"):
            line = line.strip()
            if line.startswith("ds_read"):
                reads += 1
            wait = re.search(r"lgkmcnt\((\d+)\)", line)
            if wait:
                reads = min(reads, int(wait.group(1)))
            if line.startswith("buffer_load") and line.split(";")[0].rstrip().endswith(" lds"):
                loads += 1
                worst = max(worst, reads)
        found.append((name, loads, worst))
    return found


def test_scan_sees_a_missing_wait():
    body = ["ds_read_b128 v[0:3], v9", "ds_read_b128 v[4:7], v9 offset:16", "s_waitcnt lgkmcnt(1)",
            "buffer_load_dwordx4 v8, s[0:3], 0 offen nt lds"]
    listing = "\n".join(["_Z1k:"] + ["\t" + line for line in body] + ["\ts_endpgm", ""])
    assert outstanding_reads("\n" + listing) == [("_Z1k", 1, 1)]
    assert outstanding_reads("\n" + listing.replace("lgkmcnt(1)", "lgkmcnt(0)")) == [("_Z1k", 1, 0)]


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
@pytest.mark.parametrize("source,kernels", [("gemm_layer_skinny.hip", 10), ("gemm_skinny.hip", 2)])
def test_slots_are_refilled_after_their_reads(source, kernels, tmp_path):
    out = str(tmp_path / "listing.s")
    cmd = [_hipcc(), *B.COMMON_FLAGS, *B.FILE_FLAGS.get(source, []), "-I", B.INCLUDE, "-I", B.CSRC,
           "--cuda-device-only", "-S", os.path.join(B.CSRC, source), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    found = [f for f in outstanding_reads(open(out).read()) if f[1] > 0]
    assert len(found) == kernels, found
    assert not [f for f in found if f[2] > 0], found
