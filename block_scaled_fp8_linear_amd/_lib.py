"""ctypes binding of libfp8bl.so: argument marshalling only.

Tensors are torch tensors on a HIP device; only their data pointers, sizes
and the current stream cross into the library. No arithmetic of the method
happens here. If the shared library has not been built, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import re
import struct

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libfp8bl.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG_DIR), "include", "fp8bl.h")
LAYERS_HEADER_PATH = os.path.join(os.path.dirname(_PKG_DIR), "include", "fp8bl_layers.h")
INT8_HEADER_PATH = os.path.join(os.path.dirname(_PKG_DIR), "include", "fp8bl_int8.h")
QKV_HEADER_PATH = os.path.join(os.path.dirname(_PKG_DIR), "include", "fp8bl_qkv.h")

FP8BL_OK = 0
FP8BL_INVALID_ARG = 1
FP8BL_ALIGNMENT = 2
FP8BL_WORKSPACE = 3
FP8BL_UNSUPPORTED_DEVICE = 4
FP8BL_HIP_ERROR = 5

PATH_AUTO = 0
PATH_TILED = 1
PATH_SKINNY = 2
PATH_LARGE = 3

ACT_NONE = 0
ACT_RELU = 1
ACT_SILU = 2
ACT_GELU = 3
ACT_GELU_TANH = 4

_lib = None


class Fp8blError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load() -> ctypes.CDLL:
    """Load libfp8bl.so once; raise if it is missing (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m block_scaled_fp8_linear_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, sz, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.fp8_block_abi_version.restype = c_int
    lib.fp8_block_abi_version.argtypes = []
    lib.fp8_block_status_string.restype = ctypes.c_char_p
    lib.fp8_block_status_string.argtypes = [c_int]
    lib.fp8_block_device_supported.restype = c_int
    lib.fp8_block_device_supported.argtypes = [c_int]
    lib.fp8_block_dequant.restype = c_int
    lib.fp8_block_dequant.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.fp8_block_linear_workspace_size.restype = sz
    lib.fp8_block_linear_workspace_size.argtypes = [i64, i64, i64]
    lib.fp8_block_linear.restype = c_int
    lib.fp8_block_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.fp8_block_linear_ex.restype = c_int
    lib.fp8_block_linear_ex.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, sz, c_int, vp]
    lib.fp8_block_linear_noalloc.restype = c_int
    lib.fp8_block_linear_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.fp8_block_mlp_gate_up.restype = c_int
    lib.fp8_block_mlp_gate_up.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    lib.fp8_block_mlp_gate_up_ex.restype = c_int
    lib.fp8_block_mlp_gate_up_ex.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, c_int, vp]
    lib.fp8_act_quantize.restype = c_int
    lib.fp8_act_quantize.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.fp8_block_linear_w8a8_workspace_size.restype = sz
    lib.fp8_block_linear_w8a8_workspace_size.argtypes = [i64, i64, i64]
    lib.fp8_block_linear_w8a8.restype = c_int
    lib.fp8_block_linear_w8a8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.fp8_block_linear_w8a8_ex.restype = c_int
    lib.fp8_block_linear_w8a8_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, sz, c_int, vp]
    lib.fp8_block_linear_w8a8_bf16.restype = c_int
    lib.fp8_block_linear_w8a8_bf16.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.fp8_block_quantize.restype = c_int
    lib.fp8_block_quantize.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.fp8_block_quantize_bf16.restype = c_int
    lib.fp8_block_quantize_bf16.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.fp8_block_stream_read.restype = c_int
    lib.fp8_block_stream_read.argtypes = [vp, sz, vp, c_int, vp]
    for op in ("linear_act", "linear_act_backward", "glu", "glu_backward"):
        size = getattr(lib, f"fp8_block_{op}_workspace_size")
        size.restype = sz
        size.argtypes = [i64, i64, i64]
    tail = [i64, i64, i64, c_int, vp, sz, vp]   # m, n, k, act, workspace, its bytes, stream
    for op, pointers in (("linear_act", 7), ("linear_act_backward", 7), ("glu", 8), ("glu_backward", 10)):
        call = getattr(lib, f"fp8_block_{op}")
        call.restype = c_int
        call.argtypes = [vp] * pointers + tail
    for name in ("int8_row_quantize", "int8_row_quantize_bf16"):
        call = getattr(lib, name)
        call.restype = c_int
        call.argtypes = [vp, vp, vp, i64, i64, vp]
    for name, pointers in (("int8_linear", 6), ("int8_linear_bf16", 5)):
        size, call = getattr(lib, name + "_workspace_size"), getattr(lib, name)
        size.restype = sz
        size.argtypes = [i64, i64, i64]
        call.restype = c_int
        call.argtypes = [vp] * pointers + [i64, i64, i64, vp, sz, vp]
    for name in ("fp8_qk_norm_rope", "fp8_kv_store", "fp8_kv_load", "fp8_qk_norm_rope_store"):
        call = getattr(lib, name)
        call.restype = c_int
        call.argtypes = [ctypes.c_char_p, vp]
    lib.fp8_qk_norm_rope_backward_workspace_size.restype = sz
    lib.fp8_qk_norm_rope_backward_workspace_size.argtypes = [i64, i64, i64, i64]
    lib.fp8_qk_norm_rope_backward.restype = c_int
    lib.fp8_qk_norm_rope_backward.argtypes = [ctypes.c_char_p, vp, sz, vp]
    _lib = lib
    return lib


def header_functions(path: str | None = None) -> list[str]:
    """Names of the functions a header declares (include/fp8bl.h by default)."""
    text = open(path or HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?((?:fp8|int8)_\w+)\s*\(", text, flags=re.M)


def status_string(status: int) -> str:
    return load().fp8_block_status_string(int(status)).decode()


def abi_version() -> int:
    return load().fp8_block_abi_version()


def device_supported(device: int = 0) -> bool:
    return bool(load().fp8_block_device_supported(int(device)))


def workspace_size(m: int, n: int, k: int) -> int:
    return int(load().fp8_block_linear_workspace_size(int(m), int(n), int(k)))


# Raw pointer-level calls (ints are device addresses); used by the tensor API
# below and by tests that exercise argument checking without a device.

def dequant_raw(q: int, s: int, w: int, n: int, k: int, stream: int = 0) -> int:
    return load().fp8_block_dequant(q, s, w, n, k, stream)


def linear_raw(x: int, q: int, s: int, y: int, m: int, n: int, k: int,
               ws: int, ws_bytes: int, path: int = PATH_AUTO, stream: int = 0) -> int:
    return load().fp8_block_linear_ex(x, q, s, y, m, n, k, ws, ws_bytes, path, stream)


def linear_noalloc_raw(x: int, q: int, s: int, y: int, m: int, n: int, k: int,
                       stream: int = 0) -> int:
    return load().fp8_block_linear_noalloc(x, q, s, y, m, n, k, stream)


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def mlp_gate_up_raw(x: int, qg: int, sg: int, qu: int, su: int, h: int,
                    m: int, n: int, k: int, stream: int = 0) -> int:
    return load().fp8_block_mlp_gate_up(x, qg, sg, qu, su, h, m, n, k, stream)


def mlp_gate_up_ex_raw(x: int, qg: int, sg: int, qu: int, su: int, h: int,
                       m: int, n: int, k: int, path: int, stream: int = 0) -> int:
    return load().fp8_block_mlp_gate_up_ex(x, qg, sg, qu, su, h, m, n, k, path, stream)


def act_quantize_raw(x: int, xq: int, xs: int, m: int, k: int, stream: int = 0) -> int:
    return load().fp8_act_quantize(x, xq, xs, m, k, stream)


def w8a8_workspace_size(m: int, n: int, k: int) -> int:
    return int(load().fp8_block_linear_w8a8_workspace_size(int(m), int(n), int(k)))


def linear_w8a8_raw(xq: int, xs: int, q: int, s: int, y: int, m: int, n: int, k: int,
                    ws: int, ws_bytes: int, stream: int = 0) -> int:
    return load().fp8_block_linear_w8a8(xq, xs, q, s, y, m, n, k, ws, ws_bytes, stream)


def linear_w8a8_ex_raw(xq: int, xs: int, q: int, s: int, y: int, m: int, n: int, k: int,
                       ws: int, ws_bytes: int, path: int, stream: int = 0) -> int:
    return load().fp8_block_linear_w8a8_ex(xq, xs, q, s, y, m, n, k, ws, ws_bytes, path, stream)


def linear_w8a8_bf16_raw(x: int, q: int, s: int, y: int, m: int, n: int, k: int,
                         ws: int, ws_bytes: int, stream: int = 0) -> int:
    return load().fp8_block_linear_w8a8_bf16(x, q, s, y, m, n, k, ws, ws_bytes, stream)


def quantize_raw(w: int, q: int, s: int, n: int, k: int, stream: int = 0) -> int:
    return load().fp8_block_quantize(w, q, s, n, k, stream)


def quantize_bf16_raw(w: int, q: int, s: int, n: int, k: int, stream: int = 0) -> int:
    return load().fp8_block_quantize_bf16(w, q, s, n, k, stream)


def stream_read_raw(buf: int, nbytes: int, sink: int, blocks: int, stream: int = 0) -> int:
    return load().fp8_block_stream_read(buf, nbytes, sink, blocks, stream)


# Layer operators (include/fp8bl_layers.h).

_layer_calls: dict = {}


def layer_calls(op: str) -> tuple:
    """The workspace query and the call of fp8_block_<op>."""
    got = _layer_calls.get(op)
    if got is None:
        lib = load()
        got = _layer_calls[op] = (getattr(lib, f"fp8_block_{op}_workspace_size"),
                                  getattr(lib, f"fp8_block_{op}"))
    return got


def layer_workspace_size(op: str, m: int, n: int, k: int) -> int:
    """Workspace bytes of fp8_block_<op>: linear_act, linear_act_backward, glu
    or glu_backward."""
    return int(layer_calls(op)[0](int(m), int(n), int(k)))


def linear_act_raw(x: int, q: int, s: int, bias: int, residual: int, z: int, y: int, m: int, n: int,
                   k: int, act: int, ws: int, ws_bytes: int, stream: int = 0) -> int:
    return load().fp8_block_linear_act(x, q, s, bias, residual, z, y, m, n, k, act, ws, ws_bytes,
                                       stream)


def linear_act_backward_raw(dy: int, z: int, q: int, s: int, dz: int, dbias: int, dx: int, m: int,
                            n: int, k: int, act: int, ws: int, ws_bytes: int, stream: int = 0) -> int:
    return load().fp8_block_linear_act_backward(dy, z, q, s, dz, dbias, dx, m, n, k, act, ws,
                                                ws_bytes, stream)


def glu_raw(x: int, qg: int, sg: int, qu: int, su: int, g: int, u: int, h: int, m: int, n: int, k: int,
            act: int, ws: int, ws_bytes: int, stream: int = 0) -> int:
    return load().fp8_block_glu(x, qg, sg, qu, su, g, u, h, m, n, k, act, ws, ws_bytes, stream)


def glu_backward_raw(dh: int, g: int, u: int, qg: int, sg: int, qu: int, su: int, dg: int, du: int,
                     dx: int, m: int, n: int, k: int, act: int, ws: int, ws_bytes: int,
                     stream: int = 0) -> int:
    return load().fp8_block_glu_backward(dh, g, u, qg, sg, qu, su, dg, du, dx, m, n, k, act, ws,
                                         ws_bytes, stream)


# 8-bit integer linear (include/fp8bl_int8.h).

def int8_row_quantize_raw(x: int, q: int, s: int, m: int, k: int, bf16: bool, stream: int = 0) -> int:
    lib = load()
    return (lib.int8_row_quantize_bf16 if bf16 else lib.int8_row_quantize)(x, q, s, m, k, stream)


def int8_linear_raw(xq: int, xs: int, wq: int, ws: int, bias: int, y: int, m: int, n: int, k: int,
                    work: int, work_bytes: int, stream: int = 0) -> int:
    return load().int8_linear(xq, xs, wq, ws, bias, y, m, n, k, work, work_bytes, stream)


def int8_linear_bf16_raw(x: int, wq: int, ws: int, bias: int, y: int, m: int, n: int, k: int,
                         work: int, work_bytes: int, stream: int = 0) -> int:
    return load().int8_linear_bf16(x, wq, ws, bias, y, m, n, k, work, work_bytes, stream)


def int8_workspace_size(m: int, n: int, k: int, from_bf16: bool = True) -> int:
    """Workspace bytes of int8_linear_bf16, or of int8_linear."""
    lib = load()
    size = lib.int8_linear_bf16_workspace_size if from_bf16 else lib.int8_linear_workspace_size
    return int(size(int(m), int(n), int(k)))


# From the QKV projection to its cache (include/fp8bl_qkv.h).

MAX_AXES = 8
MAX_PAIRS = 128

# struct fp8bl_qkv: its members in order, every one of eight bytes but the axes
_HEADS = ("q", "k", "v", "q_out", "k_out", "v_out", "dq", "dk")
_QKV_FIELDS = (("tokens", "q_heads", "k_heads", "head_dim")
               + tuple(f"{h}_{part}" for h in _HEADS for part in ("data", "token_stride", "head_stride"))
               + ("q_weight", "k_weight", "dq_weight", "dk_weight", "positions", "inv_freq",
                  "axes", "pairs", "interleaved", "eps",
                  "slots", "k_cache", "v_cache", "k_scale", "v_scale", "cache_rows"))
_QKV_STRUCT = struct.Struct(f"={_QKV_FIELDS.index('eps')}qd{len(_QKV_FIELDS) - _QKV_FIELDS.index('eps') - 1}q"
                            f"{MAX_PAIRS}s")
qkv_pack = _QKV_STRUCT.pack


def qkv_struct(axis: bytes = b"", **members) -> bytes:
    """struct fp8bl_qkv with the named members set and zeros elsewhere."""
    unknown = set(members) - set(_QKV_FIELDS)
    if unknown:
        raise ValueError(f"no such members: {sorted(unknown)}")
    return qkv_pack(*(members.get(f, 0) for f in _QKV_FIELDS), axis)


def qk_norm_rope_raw(args: bytes, stream: int = 0) -> int:
    return load().fp8_qk_norm_rope(args, stream)


def qk_norm_rope_backward_raw(args: bytes, work: int, work_bytes: int, stream: int = 0) -> int:
    return load().fp8_qk_norm_rope_backward(args, work, work_bytes, stream)


def qk_norm_rope_backward_workspace_size(tokens: int, q_heads: int, k_heads: int, head_dim: int) -> int:
    return int(load().fp8_qk_norm_rope_backward_workspace_size(int(tokens), int(q_heads), int(k_heads),
                                                               int(head_dim)))


def kv_store_raw(args: bytes, stream: int = 0) -> int:
    return load().fp8_kv_store(args, stream)


def kv_load_raw(args: bytes, stream: int = 0) -> int:
    return load().fp8_kv_load(args, stream)


def qk_norm_rope_store_raw(args: bytes, stream: int = 0) -> int:
    return load().fp8_qk_norm_rope_store(args, stream)
