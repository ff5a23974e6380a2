"""Build libfp8bl.so (gfx950 only) and the compiled part of the binding in-tree.

    python -m block_scaled_fp8_linear_amd.build

Each HIP source is compiled to an object in ``_build/`` (in parallel), then
linked into ``block_scaled_fp8_linear_amd/libfp8bl.so``; binding/tensors.cpp, host
code over torch's headers, becomes ``_tensors.so`` beside it. Always rebuilds.

The library needs hipcc alone: it is linked first, whatever becomes of the binding.
Without torch (run this file by its path then) there is no binding to build.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libfp8bl.so")
BINDING = os.path.join(PKG_DIR, "binding", "tensors.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_tensors.so")

ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libfp8bl.so)")


COMMON_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fvisibility=hidden",
    # The dequant is a multiply followed by a rounding; keep every fp op as written.
    "-ffp-contract=off",
    # Packed fp32 VALU forms stay off (scalar fp32 only).
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


# Per-file device code generation options. The W8A8 large-tile kernel keeps
# its 192 accumulators in VGPRs and scales each MFMA block sum with a VALU
# FMA: the VGPR form of the MFMA puts those sums where the FMA can read them
# (the default AGPR form costs a copy per value, doubling the VALU work).
FILE_FLAGS = {
    "gemm_w8a8_large.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
}


def _compile(src: str, obj: str, verbose: bool) -> None:
    extra = FILE_FLAGS.get(os.path.basename(src), [])
    cmd = [hipcc(), *COMMON_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _rocm_dir() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))


def _cxx() -> str:
    """The host's C++ compiler, or the one that hipcc drives."""
    for cand in ("g++", "c++", "clang++"):
        if shutil.which(cand):
            return cand
    return os.path.join(_rocm_dir(), "llvm", "bin", "clang++")


def _compile_binding(torch_dir: str, obj: str, verbose: bool) -> None:
    """binding/tensors.cpp to an object: host code only, with the host compiler."""
    rocm = _rocm_dir()
    includes = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), os.path.join(rocm, "include"), INCLUDE]
    cmd = [_cxx(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__", "-c", BINDING, "-o", obj]
    for path in includes:
        cmd += ["-I", path]
    _run(cmd, "compilation of tensors.cpp", verbose)


def _link_binding(torch_dir: str, obj: str, verbose: bool) -> None:
    """Against the library beside it and torch, which is loaded by then."""
    torch_lib = os.path.join(torch_dir, "lib")
    tmp = BINDING_PATH + ".tmp"
    _run([_cxx(), "-shared", obj, "-o", tmp, "-L", PKG_DIR, "-l:libfp8bl.so", "-L", torch_lib, "-lc10", "-ltorch_cpu",
          "-ltorch_hip", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "link of _tensors.so", verbose)
    os.replace(tmp, BINDING_PATH)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    objs = [os.path.join(BUILD_DIR, os.path.basename(s) + ".o") for s in srcs]
    binding, torch_dir = os.path.join(BUILD_DIR, "tensors.cpp.o"), _torch_dir()
    host = None
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        if torch_dir is not None:
            host = ex.submit(_compile_binding, torch_dir, binding, verbose)
        list(ex.map(lambda so: _compile(so[0], so[1], verbose), zip(srcs, objs)))
    tmp = LIB_PATH + ".tmp"
    _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp], "link", verbose)
    os.replace(tmp, LIB_PATH)
    if host is None:
        print("no torch here: _tensors.so, the compiled binding over it, is not built", file=sys.stderr)
        return LIB_PATH
    host.result()
    _link_binding(torch_dir, binding, verbose)
    return LIB_PATH


if __name__ == "__main__":
    path = build(verbose="-v" in sys.argv)
    print(path)
