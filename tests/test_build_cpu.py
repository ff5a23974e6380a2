"""The build's order: the C library needs hipcc alone and is there whatever becomes
of the binding over torch. Nothing is compiled here."""

from __future__ import annotations

import importlib.util
import os
import runpy
import subprocess
import sys

import pytest

pytest.importorskip("torch")

from block_scaled_fp8_linear_amd import build as B  # noqa: E402


@pytest.fixture
def dry(monkeypatch, tmp_path):
    """Commands are recorded and leave an empty output; `fail` makes one fail."""
    ran, fail = [], []

    def run(cmd, **kw):
        ran.append(cmd)
        if any(f in cmd for f in fail):
            return subprocess.CompletedProcess(cmd, 1, "", "failed")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "hipcc", lambda: "/opt/rocm/bin/hipcc")
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libfp8bl.so"))
    monkeypatch.setattr(B, "BINDING_PATH", str(tmp_path / "_tensors.so"))
    return ran, fail


def without(monkeypatch, name):
    find = importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda n, *a: None if n == name else find(n, *a))


def test_both_are_built(dry):
    B.build()
    assert os.path.exists(B.LIB_PATH) and os.path.exists(B.BINDING_PATH)


def test_without_torch_the_library_is_built(dry, monkeypatch, capsys):
    without(monkeypatch, "torch")
    assert B.build() == B.LIB_PATH
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.BINDING_PATH)
    assert all(cmd[0] == "/opt/rocm/bin/hipcc" for cmd in dry[0])
    assert "_tensors.so" in capsys.readouterr().err


def test_a_binding_that_fails_leaves_the_library(dry):
    dry[1].append(B.BINDING)
    with pytest.raises(RuntimeError, match="tensors.cpp"):
        B.build()
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.BINDING_PATH)


def test_without_a_host_compiler_the_one_of_hipcc_is_taken(dry, monkeypatch):
    monkeypatch.setattr(B.shutil, "which", lambda name: None)
    B.build()
    host = [cmd[0] for cmd in dry[0] if cmd[0] != "/opt/rocm/bin/hipcc"]
    assert len(host) == 2 and all(c.endswith(os.path.join("llvm", "bin", "clang++")) for c in host)


def test_the_file_runs_by_its_path(dry, monkeypatch, capsys):
    """Without torch the package itself cannot be imported: the file runs alone."""
    without(monkeypatch, "torch")
    monkeypatch.setattr(sys, "argv", ["build.py"])
    module = runpy.run_path(B.__file__, run_name="alone")
    assert module["_torch_dir"]() is None and callable(module["build"])
