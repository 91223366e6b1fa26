"""BitLinear W1.58A8 on MI355X (gfx950): thin Python binding of ``libbitlinear.so``.

The layer is the BitNet b1.58 BitLinear (bako.co, "The BitLinear Layer and
AbsMean Quantization"; deepmox.com chapter 8, "A low-bit model is a whole-stack
design"): absmean-ternarized weights packed at 2 bits, per-token absmax int8
activations, int32 accumulation and a bf16 rescale.  Every step runs in the HIP
kernels behind the C ABI (``include/bitlinear.h``); this module only marshals
torch tensors (device memory, the current stream) into those calls.  There is
no fallback: if the library is missing, importing raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from ._build import LIB_PATH, INCLUDE

__all__ = [
    "BitLinearError", "bl_packed_bytes", "bl_ternarize_pack_workspace_bytes", "bl_ternarize_pack",
    "bl_quant_act", "bl_linear", "bl_bitlinear", "bl_unpack_ternary", "bl_status_string", "library", "declared_symbols",
    "bl_ternarize_pack_glu", "bl_linear_glu", "bl_bitlinear_glu", "bl_pack_transposed", "bl_bitlinear_backward_x",
    "bl_backward_w_workspace_bytes", "bl_bitlinear_backward_w", "bl_ternarize_pack_noalloc",
    "bl_packed_bytes_b3", "bl_ternarize_pack_b3", "bl_bitlinear_b3",
    "bl_rmsnorm_quant", "bl_rmsnorm_backward_workspace_bytes", "bl_rmsnorm_backward", "bl_rope_frequencies", "bl_rope",
    "Rope", "KVCache", "KVBatch", "bl_kv_append", "bl_kv_read", "bl_attention_workspace_bytes", "bl_attention",
]


class BitLinearError(RuntimeError):
    """A ``bl_*`` call returned a status other than BL_OK."""

    def __init__(self, func: str, status: int):
        super().__init__(f"{func}: {bl_status_string(status)} ({status})")
        self.status = status


# BITLINEAR_LIB may name another build of the same library (the test suite
# loads a host-sanitizer build this way); by default the in-tree build.
_LIB_FILE = os.environ.get("BITLINEAR_LIB") or LIB_PATH
if not os.path.exists(_LIB_FILE):
    raise ImportError(f"libbitlinear.so is not built ({_LIB_FILE}); run __graft_entry__.build()")

_lib = ctypes.CDLL(_LIB_FILE)
_P, _I64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_lib.bl_packed_bytes.argtypes = [_I64, _I64]
_lib.bl_packed_bytes.restype = _SZ
_lib.bl_ternarize_pack_workspace_bytes.argtypes = [_I64, _I64]
_lib.bl_ternarize_pack_workspace_bytes.restype = _SZ
_lib.bl_ternarize_pack.argtypes = [_P, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.bl_ternarize_pack.restype = ctypes.c_int
_lib.bl_ternarize_pack_noalloc.argtypes = [_P, _I64, _I64, _P, _P, _P]
_lib.bl_ternarize_pack_noalloc.restype = ctypes.c_int
_lib.bl_packed_bytes_b3.argtypes = [_I64, _I64]
_lib.bl_packed_bytes_b3.restype = _SZ
_lib.bl_ternarize_pack_b3.argtypes = [_P, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.bl_ternarize_pack_b3.restype = ctypes.c_int
_lib.bl_bitlinear_b3.argtypes = [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P]
_lib.bl_bitlinear_b3.restype = ctypes.c_int
_lib.bl_quant_act.argtypes = [_P, _I64, _I64, _P, _P, _P]
_lib.bl_quant_act.restype = ctypes.c_int
_lib.bl_linear.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P]
_lib.bl_linear.restype = ctypes.c_int
_lib.bl_bitlinear.argtypes = [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P]
_lib.bl_bitlinear.restype = ctypes.c_int
_lib.bl_unpack_ternary.argtypes = [_P, _I64, _I64, _P, _P]
_lib.bl_ternarize_pack_glu.argtypes = [_P, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.bl_ternarize_pack_glu.restype = ctypes.c_int
_lib.bl_linear_glu.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _P, _P]
_lib.bl_linear_glu.restype = ctypes.c_int
_lib.bl_bitlinear_glu.argtypes = [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P]
_lib.bl_bitlinear_glu.restype = ctypes.c_int
_lib.bl_pack_transposed.argtypes = [_P, _I64, _I64, _P, _P]
_lib.bl_pack_transposed.restype = ctypes.c_int
_lib.bl_bitlinear_backward_x.argtypes = [_P, _P, _P, _I64, _I64, _I64, _P, _P]
_lib.bl_bitlinear_backward_x.restype = ctypes.c_int
_lib.bl_backward_w_workspace_bytes.argtypes = [_I64, _I64, _I64]
_lib.bl_backward_w_workspace_bytes.restype = _SZ
_lib.bl_bitlinear_backward_w.argtypes = [_P, _P, _P, _I64, _I64, _I64, _P, _P, _SZ, _P]
_lib.bl_bitlinear_backward_w.restype = ctypes.c_int
_lib.bl_unpack_ternary.restype = ctypes.c_int
_F32, _F64, _INT = ctypes.c_float, ctypes.c_double, ctypes.c_int
_lib.bl_rmsnorm_quant.argtypes = [_P, _P, _P, _I64, _I64, _F32, _P, _P, _P, _P, _P, _P]
_lib.bl_rmsnorm_quant.restype = _INT
_lib.bl_rmsnorm_backward_workspace_bytes.argtypes = [_I64, _I64]
_lib.bl_rmsnorm_backward_workspace_bytes.restype = _SZ
_lib.bl_rmsnorm_backward.argtypes = [_P, _P, _P, _P, _I64, _I64, _F32, _P, _P, _P, _SZ, _P]
_lib.bl_rmsnorm_backward.restype = _INT
_lib.bl_rope_frequencies.argtypes = [_I64, _F64, _INT, _F64, _F64, _F64, _F64, _P]
_lib.bl_rope_frequencies.restype = _INT
_lib.bl_rope.argtypes = [_P, _I64, _I64, _P, _P, _I64, _I64, _I64, _INT, _P, _I64, _I64, _P]
_lib.bl_rope.restype = _INT
_lib.bl_kv_append.argtypes = [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _I64, _P, _P]
_lib.bl_kv_append.restype = _INT
_lib.bl_kv_read.argtypes = [_P, _P, _P, _P, _P]
_lib.bl_kv_read.restype = _INT
_lib.bl_attention_workspace_bytes.argtypes = [_P, _P, _I64]
_lib.bl_attention_workspace_bytes.restype = _SZ
_lib.bl_attention.argtypes = [_P, _P, _P, _I64, _I64, _I64, _F32, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.bl_attention.restype = _INT
_lib.bl_status_string.argtypes = [ctypes.c_int]
_lib.bl_status_string.restype = ctypes.c_char_p


def library() -> ctypes.CDLL:
    """The loaded C-ABI library (for callers that marshal pointers themselves)."""
    return _lib


def declared_symbols() -> list[str]:
    """Names of the functions declared in ``include/bitlinear.h``."""
    with open(os.path.join(INCLUDE, "bitlinear.h")) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bl_\w+)\s*\(", text)))


def bl_status_string(status: int) -> str:
    return _lib.bl_status_string(int(status)).decode()


def _check(func: str, status: int) -> None:
    if status != 0:
        raise BitLinearError(func, status)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object around it: 0.1 us instead
# of 2 us, of a call that takes about 4 us in the library.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(device: torch.device) -> int:
    return _raw_stream(device.index)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple | None = None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def bl_packed_bytes(n: int, k: int) -> int:
    return int(_lib.bl_packed_bytes(n, k))


def bl_ternarize_pack_workspace_bytes(n: int, k: int) -> int:
    return int(_lib.bl_ternarize_pack_workspace_bytes(n, k))


def bl_ternarize_pack(w: torch.Tensor, packed: torch.Tensor | None = None, gamma: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None):
    """fp32 weights ``[n][k]`` -> (packed uint8 [bl_packed_bytes], gamma fp32 [1])."""
    _need(w, "w", torch.float32)
    n, k = w.shape
    nbytes = bl_packed_bytes(n, k)
    if packed is None:
        packed = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=w.device)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=w.device)
    ws = bl_ternarize_pack_workspace_bytes(n, k)
    if workspace is None:
        workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=w.device)
    _check("bl_ternarize_pack", _lib.bl_ternarize_pack(_ptr(w), n, k, _ptr(packed), _ptr(gamma), _ptr(workspace),
                                                       workspace.numel(), _stream(w.device)))
    return packed, gamma


def bl_ternarize_pack_noalloc(w: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor):
    """bl_ternarize_pack into caller-provided outputs, with the library's static
    device bins instead of a workspace (the call itself allocates nothing)."""
    _need(w, "w", torch.float32)
    n, k = w.shape
    _need(packed, "packed", torch.uint8)
    _need(gamma, "gamma", torch.float32)
    if packed.numel() < bl_packed_bytes(n, k) or gamma.numel() < 1:
        raise ValueError("packed or gamma buffer too small")
    _check("bl_ternarize_pack_noalloc", _lib.bl_ternarize_pack_noalloc(_ptr(w), n, k, _ptr(packed), _ptr(gamma),
                                                                       _stream(w.device)))
    return packed, gamma


def bl_packed_bytes_b3(n: int, k: int) -> int:
    return int(_lib.bl_packed_bytes_b3(n, k))


def bl_ternarize_pack_b3(w: torch.Tensor, packed: torch.Tensor | None = None, gamma: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None):
    """fp32 weights ``[n][k]`` -> (five-trits-per-byte uint8 [bl_packed_bytes_b3], gamma fp32 [1])."""
    _need(w, "w", torch.float32)
    n, k = w.shape
    if packed is None:
        packed = torch.empty(max(bl_packed_bytes_b3(n, k), 1), dtype=torch.uint8, device=w.device)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=w.device)
    if workspace is None:
        workspace = torch.empty(max(bl_ternarize_pack_workspace_bytes(n, k), 16), dtype=torch.uint8, device=w.device)
    _check("bl_ternarize_pack_b3", _lib.bl_ternarize_pack_b3(_ptr(w), n, k, _ptr(packed), _ptr(gamma),
                                                             _ptr(workspace), workspace.numel(), _stream(w.device)))
    return packed, gamma


def bl_bitlinear_b3(packed: torch.Tensor, gamma: torch.Tensor, x: torch.Tensor, n: int,
                    xq: torch.Tensor | None = None, alpha: torch.Tensor | None = None,
                    acc: torch.Tensor | None | bool = True, y: torch.Tensor | None | bool = True):
    """bf16 activations ``[m][k]`` through the layer with five-trits-per-byte
    weights: returns (acc or None, y or None, xq, alpha)."""
    _need(x, "x", torch.bfloat16)
    m, k = x.shape
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=dev)
    if alpha is None:
        alpha = torch.empty(m, dtype=torch.float32, device=dev)
    _need(xq, "xq", torch.int8, (m, k))
    _need(alpha, "alpha", torch.float32, (m,))
    if acc is True:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    if y is True:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    acc = acc if isinstance(acc, torch.Tensor) else None
    y = y if isinstance(y, torch.Tensor) else None
    if acc is not None:
        _need(acc, "acc", torch.int32, (m, n))
    if y is not None:
        _need(y, "y", torch.bfloat16, (m, n))
    _need(packed, "packed", torch.uint8)
    if packed.numel() < bl_packed_bytes_b3(n, k):
        raise ValueError("packed buffer is smaller than bl_packed_bytes_b3(n, k)")
    _check("bl_bitlinear_b3", _lib.bl_bitlinear_b3(_ptr(packed), _ptr(gamma), _ptr(x), m, n, k, _ptr(xq),
                                                   _ptr(alpha), _ptr(acc), _ptr(y), _stream(dev)))
    return acc, y, xq, alpha


def bl_quant_act(x: torch.Tensor, xq: torch.Tensor | None = None, alpha: torch.Tensor | None = None):
    """bf16 activations ``[m][k]`` -> (int8 [m][k], per-token absmax fp32 [m])."""
    _need(x, "x", torch.bfloat16)
    m, k = x.shape
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=x.device)
    if alpha is None:
        alpha = torch.empty(m, dtype=torch.float32, device=x.device)
    _need(xq, "xq", torch.int8, (m, k))
    _need(alpha, "alpha", torch.float32, (m,))
    _check("bl_quant_act", _lib.bl_quant_act(_ptr(x), m, k, _ptr(xq), _ptr(alpha), _stream(x.device)))
    return xq, alpha


def bl_linear(packed: torch.Tensor, gamma: torch.Tensor, xq: torch.Tensor, alpha: torch.Tensor, n: int,
              acc: torch.Tensor | None | bool = True, y: torch.Tensor | None | bool = True):
    """Packed ternary ``[n][k]`` times int8 ``[m][k]`` -> (int32 acc [m][n] or None, bf16 y [m][n] or None).

    ``acc``/``y``: a tensor to write into, True to allocate, or False/None to skip."""
    _need(xq, "xq", torch.int8)
    m, k = xq.shape
    dev = xq.device
    if acc is True:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    if y is True:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    acc = acc if isinstance(acc, torch.Tensor) else None
    y = y if isinstance(y, torch.Tensor) else None
    if acc is not None:
        _need(acc, "acc", torch.int32, (m, n))
    if y is not None:
        _need(y, "y", torch.bfloat16, (m, n))
    _need(packed, "packed", torch.uint8)
    if packed.numel() < bl_packed_bytes(n, k):
        raise ValueError("packed buffer is smaller than bl_packed_bytes(n, k)")
    _check("bl_linear", _lib.bl_linear(_ptr(packed), _ptr(gamma), _ptr(xq), _ptr(alpha), m, n, k, _ptr(acc), _ptr(y),
                                       _stream(dev)))
    return acc, y


def bl_bitlinear(packed: torch.Tensor, gamma: torch.Tensor, x: torch.Tensor, n: int,
                 xq: torch.Tensor | None = None, alpha: torch.Tensor | None = None,
                 acc: torch.Tensor | None | bool = True, y: torch.Tensor | None | bool = True):
    """bf16 activations ``[m][k]`` through the whole layer in one call:
    returns (acc or None, y or None, xq, alpha)."""
    _need(x, "x", torch.bfloat16)
    m, k = x.shape
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=dev)
    if alpha is None:
        alpha = torch.empty(m, dtype=torch.float32, device=dev)
    _need(xq, "xq", torch.int8, (m, k))
    _need(alpha, "alpha", torch.float32, (m,))
    if acc is True:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    if y is True:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    acc = acc if isinstance(acc, torch.Tensor) else None
    y = y if isinstance(y, torch.Tensor) else None
    if acc is not None:
        _need(acc, "acc", torch.int32, (m, n))
    if y is not None:
        _need(y, "y", torch.bfloat16, (m, n))
    _need(packed, "packed", torch.uint8)
    if packed.numel() < bl_packed_bytes(n, k):
        raise ValueError("packed buffer is smaller than bl_packed_bytes(n, k)")
    _check("bl_bitlinear", _lib.bl_bitlinear(_ptr(packed), _ptr(gamma), _ptr(x), m, n, k, _ptr(xq), _ptr(alpha),
                                             _ptr(acc), _ptr(y), _stream(dev)))
    return acc, y, xq, alpha


def bl_ternarize_pack_glu(w: torch.Tensor, packed: torch.Tensor | None = None, gamma: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None):
    """fp32 gate+up weights ``[2f][k]`` (gate rows first) -> (packed with
    alternating gate/up row tiles, gamma fp32 [1])."""
    _need(w, "w", torch.float32)
    n2, k = w.shape
    f = n2 // 2
    nbytes = bl_packed_bytes(n2, k)
    if packed is None:
        packed = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=w.device)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=w.device)
    ws = bl_ternarize_pack_workspace_bytes(n2, k)
    if workspace is None:
        workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=w.device)
    if n2 % 2:
        raise ValueError("a gate+up matrix has an even number of rows")
    _check("bl_ternarize_pack_glu", _lib.bl_ternarize_pack_glu(_ptr(w), f, k, _ptr(packed), _ptr(gamma),
                                                               _ptr(workspace), workspace.numel(), _stream(w.device)))
    return packed, gamma


def bl_linear_glu(packed: torch.Tensor, gamma: torch.Tensor, xq: torch.Tensor, alpha: torch.Tensor, f: int,
                  h: torch.Tensor | None = None) -> torch.Tensor:
    """Gated product from int8 activations ``[m][k]``: h bf16 [m][f]."""
    _need(xq, "xq", torch.int8)
    m, k = xq.shape
    if h is None:
        h = torch.empty((m, f), dtype=torch.bfloat16, device=xq.device)
    _need(h, "h", torch.bfloat16, (m, f))
    _need(packed, "packed", torch.uint8)
    if packed.numel() < bl_packed_bytes(2 * f, k):
        raise ValueError("packed buffer is smaller than bl_packed_bytes(2f, k)")
    _check("bl_linear_glu", _lib.bl_linear_glu(_ptr(packed), _ptr(gamma), _ptr(xq), _ptr(alpha), m, f, k, _ptr(h),
                                               _stream(xq.device)))
    return h


def bl_bitlinear_glu(packed: torch.Tensor, gamma: torch.Tensor, x: torch.Tensor, f: int,
                     xq: torch.Tensor | None = None, alpha: torch.Tensor | None = None,
                     h: torch.Tensor | None = None):
    """bf16 activations ``[m][k]`` through quantization, the gate+up product
    and squared-ReLU gating: returns (h bf16 [m][f], xq, alpha)."""
    _need(x, "x", torch.bfloat16)
    m, k = x.shape
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=dev)
    if alpha is None:
        alpha = torch.empty(m, dtype=torch.float32, device=dev)
    if h is None:
        h = torch.empty((m, f), dtype=torch.bfloat16, device=dev)
    _need(xq, "xq", torch.int8, (m, k))
    _need(alpha, "alpha", torch.float32, (m,))
    _need(h, "h", torch.bfloat16, (m, f))
    _need(packed, "packed", torch.uint8)
    if packed.numel() < bl_packed_bytes(2 * f, k):
        raise ValueError("packed buffer is smaller than bl_packed_bytes(2f, k)")
    _check("bl_bitlinear_glu", _lib.bl_bitlinear_glu(_ptr(packed), _ptr(gamma), _ptr(x), m, f, k, _ptr(xq),
                                                     _ptr(alpha), _ptr(h), _stream(dev)))
    return h, xq, alpha


def bl_pack_transposed(packed: torch.Tensor, n: int, k: int, packed_t: torch.Tensor | None = None) -> torch.Tensor:
    """Packed q ``[n][k]`` -> packed q^T ``[k][n]`` (n % 64 == 0)."""
    _need(packed, "packed", torch.uint8)
    if packed.numel() < bl_packed_bytes(n, k):
        raise ValueError("packed buffer is smaller than bl_packed_bytes(n, k)")
    if packed_t is None:
        packed_t = torch.empty(max(bl_packed_bytes(k, n), 1), dtype=torch.uint8, device=packed.device)
    _check("bl_pack_transposed", _lib.bl_pack_transposed(_ptr(packed), n, k, _ptr(packed_t), _stream(packed.device)))
    return packed_t


def bl_bitlinear_backward_x(packed_t: torch.Tensor, gamma: torch.Tensor, dy: torch.Tensor, k: int,
                            dx: torch.Tensor | None = None) -> torch.Tensor:
    """Straight-through input gradient: dx fp32 [m][k] = gamma * dy q, from
    packed q^T (bl_pack_transposed) and dy bf16 [m][n]."""
    _need(dy, "dy", torch.bfloat16)
    m, n = dy.shape
    if dx is None:
        dx = torch.empty((m, k), dtype=torch.float32, device=dy.device)
    _need(dx, "dx", torch.float32, (m, k))
    _need(packed_t, "packed_t", torch.uint8)
    if packed_t.numel() < bl_packed_bytes(k, n):
        raise ValueError("packed_t buffer is smaller than bl_packed_bytes(k, n)")
    _check("bl_bitlinear_backward_x", _lib.bl_bitlinear_backward_x(_ptr(packed_t), _ptr(gamma), _ptr(dy), m, n, k,
                                                                   _ptr(dx), _stream(dy.device)))
    return dx


def bl_backward_w_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(_lib.bl_backward_w_workspace_bytes(m, n, k))


def bl_bitlinear_backward_w(dy: torch.Tensor, xq: torch.Tensor, alpha: torch.Tensor, dw: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Straight-through weight gradient: dw fp32 [n][k] = dy^T (alpha / 127 xq)."""
    _need(dy, "dy", torch.bfloat16)
    _need(xq, "xq", torch.int8)
    m, n = dy.shape
    k = xq.shape[1]
    _need(alpha, "alpha", torch.float32, (m,))
    if dw is None:
        dw = torch.empty((n, k), dtype=torch.float32, device=dy.device)
    _need(dw, "dw", torch.float32, (n, k))
    ws = bl_backward_w_workspace_bytes(m, n, k)
    if workspace is None:
        workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=dy.device)
    _check("bl_bitlinear_backward_w", _lib.bl_bitlinear_backward_w(_ptr(dy), _ptr(xq), _ptr(alpha), m, n, k, _ptr(dw),
                                                                   _ptr(workspace), workspace.numel(),
                                                                   _stream(dy.device)))
    return dw


def bl_unpack_ternary(packed: torch.Tensor, n: int, k: int, q: torch.Tensor | None = None) -> torch.Tensor:
    """Packed buffer -> int8 trits ``[n][k]``."""
    _need(packed, "packed", torch.uint8)
    if q is None:
        q = torch.empty((n, k), dtype=torch.int8, device=packed.device)
    _check("bl_unpack_ternary", _lib.bl_unpack_ternary(_ptr(packed), n, k, _ptr(q), _stream(packed.device)))
    return q


# ---- around the BitLinear layers ----

def _dense(t: torch.Tensor | None, name: str, dtype: torch.dtype, shape: tuple) -> int | None:
    """Address of a dense device tensor of this type and shape (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        _need(t, name, dtype, shape)
    return t.data_ptr()


def _bytes(workspace: torch.Tensor) -> int:
    """Size of a dense device tensor that a call may use as it likes."""
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return workspace.nbytes


def _heads(t: torch.Tensor, name: str, shape: tuple) -> tuple[int, int, int]:
    """Address and (token, head) strides of bf16 ``[tokens][heads][dim]`` whose last axis is adjacent."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    token, head, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    # the stride of an axis of one element is any number, and not used
    return t.data_ptr(), 0 if shape[0] == 1 else token, 0 if shape[1] == 1 else head


def bl_rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None,
                     r: torch.Tensor | None | bool = None, y: torch.Tensor | None | bool = None,
                     xhat: torch.Tensor | None | bool = None, xq: torch.Tensor | None | bool = True,
                     alpha: torch.Tensor | None = None):
    """RMS norm of ``x + residual`` (bf16 ``[m][k]``) with int8 output for bl_linear:
    returns (xq, alpha, r, y, xhat), None where an output is not asked for.

    ``r`` (the bf16 sum), ``y`` (the bf16 norm), ``xhat`` (bf16 of what the codes stand for), ``xq``: a tensor to
    write into, True to allocate, or False/None to skip; ``r`` is allocated by default if there is a residual."""
    _need(x, "x", torch.bfloat16)
    shape = m, k = x.shape
    dev = x.device
    if r is None:
        r = residual is not None
    # one at a time: a generator over them takes 0.4 us of a call of 7
    r = torch.empty_like(x) if r is True else None if r is False else r
    y = torch.empty_like(x) if y is True else None if y is False else y
    xhat = torch.empty_like(x) if xhat is True else None if xhat is False else xhat
    xq = torch.empty(shape, dtype=torch.int8, device=dev) if xq is True else None if xq is False else xq
    if xq is None:
        alpha = None
    elif alpha is None:
        alpha = torch.empty(m, dtype=torch.float32, device=dev)
    _check("bl_rmsnorm_quant", _lib.bl_rmsnorm_quant(
        x.data_ptr(), _dense(residual, "residual", torch.bfloat16, shape), _dense(weight, "weight", torch.float32, (k,)),
        m, k, eps, _dense(r, "r", torch.bfloat16, shape), _dense(y, "y", torch.bfloat16, shape),
        _dense(xhat, "xhat", torch.bfloat16, shape), _dense(xq, "xq", torch.int8, shape),
        _dense(alpha, "alpha", torch.float32, (m,)), _stream(dev)))
    return xq, alpha, r, y, xhat


def bl_rmsnorm_backward_workspace_bytes(m: int, k: int) -> int:
    return int(_lib.bl_rmsnorm_backward_workspace_bytes(m, k))


def bl_rmsnorm_backward(dn: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                        dr: torch.Tensor | None = None, dx: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None):
    """Gradients of bl_rmsnorm_quant: fp32 ``dn`` (of the norm's output) and bf16 ``dr`` (of the sum, past the
    norm; optional) -> (dx bf16 [m][k], dw fp32 [k])."""
    _need(dn, "dn", torch.float32)
    shape = m, k = dn.shape
    dev = dn.device
    if dx is None:
        dx = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if dw is None:
        dw = torch.empty(k, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(bl_rmsnorm_backward_workspace_bytes(m, k), 16), dtype=torch.uint8, device=dev)
    _check("bl_rmsnorm_backward", _lib.bl_rmsnorm_backward(
        dn.data_ptr(), _dense(r, "r", torch.bfloat16, shape), _dense(weight, "weight", torch.float32, (k,)),
        _dense(dr, "dr", torch.bfloat16, shape), m, k, eps, _dense(dx, "dx", torch.bfloat16, shape),
        _dense(dw, "dw", torch.float32, (k,)), workspace.data_ptr(), _bytes(workspace), _stream(dev)))
    return dx, dw


_ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "blend": 3}


def bl_rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                        original: float = 0.0, fast: float = 32.0, slow: float = 1.0) -> torch.Tensor:
    """Table of rotary frequencies, fp32 ``[rot / 2][2]`` on the host; ``scaling`` is "plain", "linear", "base" or
    "blend" (BL_ROPE_* of the header; ``original``, ``fast`` and ``slow`` belong to "blend")."""
    turns = torch.empty((max(rot // 2, 1), 2), dtype=torch.float32)
    _check("bl_rope_frequencies", _lib.bl_rope_frequencies(rot, base, _ROPE_SCALINGS[scaling], factor, original, fast,
                                                           slow, turns.data_ptr()))
    return turns


class Rope:
    """Rotary positions: a frequency table on the device (``bl_rope_frequencies(...).to(device)``, fp32
    ``[rot / 2][2]``), the layout of pairs and a magnitude that multiplies the result."""

    class _Struct(ctypes.Structure):
        _fields_ = [("turns", _P), ("rot", _I64), ("interleaved", ctypes.c_int32), ("magnitude", _F32)]

    def __init__(self, turns: torch.Tensor, interleaved: bool = False, magnitude: float = 1.0):
        _need(turns, "turns", torch.float32)
        if turns.dim() != 2 or turns.shape[1] != 2:
            raise ValueError(f"turns must have shape (rot / 2, 2), got {tuple(turns.shape)}")
        self.turns = turns
        self.struct = Rope._Struct(turns.data_ptr(), 2 * turns.shape[0], int(interleaved), magnitude)
        self.address = ctypes.addressof(self.struct)


def bl_rope(x: torch.Tensor, position: torch.Tensor, rope: Rope, inverse: bool = False,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 heads ``[tokens][heads][dim]`` (the last axis adjacent) rotated by their int32 positions ``[tokens]``;
    ``inverse`` gives the gradient's direction; ``out`` may be ``x``."""
    tokens, heads, dim = shape = x.shape
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    xp, xt, xh = _heads(x, "x", shape)
    yp, yt, yh = _heads(out, "out", shape)
    _check("bl_rope", _lib.bl_rope(xp, xt, xh, _dense(position, "position", torch.int32, (tokens,)), rope.address, tokens,
                                   heads, dim, int(inverse), yp, yt, yh, _stream(x.device)))
    return out


class KVCache:
    """Key/value cache in 8 bits: int8 ``k``, ``v`` [pages][heads][page_tokens][dim] and fp32 ``k_absmax``,
    ``v_absmax`` [pages][heads].  Holds the tensors that it is given."""

    class _Struct(ctypes.Structure):
        _fields_ = [("k", _P), ("v", _P), ("k_absmax", _P), ("v_absmax", _P), ("pages", _I64),
                    ("heads", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("dim", ctypes.c_int32)]

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_absmax: torch.Tensor, v_absmax: torch.Tensor):
        _need(k, "k", torch.int8)
        if k.dim() != 4:
            raise ValueError(f"k must have shape (pages, heads, page_tokens, dim), got {tuple(k.shape)}")
        _need(v, "v", torch.int8, k.shape)
        _need(k_absmax, "k_absmax", torch.float32, k.shape[:2])
        _need(v_absmax, "v_absmax", torch.float32, k.shape[:2])
        self.k, self.v, self.k_absmax, self.v_absmax = k, v, k_absmax, v_absmax
        self.pages, self.heads, self.page_tokens, self.dim = k.shape
        self.struct = KVCache._Struct(k.data_ptr(), v.data_ptr(), k_absmax.data_ptr(), v_absmax.data_ptr(), *k.shape)
        self.address = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, pages: int, heads: int, page_tokens: int, dim: int, device) -> "KVCache":
        """A cache of its own, zeroed."""
        k = torch.zeros((pages, heads, page_tokens, dim), dtype=torch.int8, device=device)
        a = torch.zeros((pages, heads), dtype=torch.float32, device=device)
        return cls(k, torch.zeros_like(k), a, torch.zeros_like(a))


class KVBatch:
    """The tokens of one step: int32 device tensors ``page_table`` [seqs][stride], ``start`` [seqs] (tokens that
    each sequence had before) and ``offsets`` [seqs + 1] (where its new tokens begin among the step's ``tokens``);
    ``max_new`` and ``max_len`` bound a sequence's new tokens and its length with them (attention sees no position
    from ``max_len`` on)."""

    class _Struct(ctypes.Structure):
        _fields_ = [("page_table", _P), ("start", _P), ("offsets", _P), ("seqs", _I64), ("table_stride", _I64),
                    ("tokens", _I64), ("max_new", _I64), ("max_len", _I64)]

    def __init__(self, page_table: torch.Tensor, start: torch.Tensor, offsets: torch.Tensor, tokens: int, max_new: int,
                 max_len: int):
        _need(page_table, "page_table", torch.int32)
        if page_table.dim() != 2:
            raise ValueError(f"page_table must have shape (seqs, stride), got {tuple(page_table.shape)}")
        seqs, stride = page_table.shape
        _need(start, "start", torch.int32, (seqs,))
        _need(offsets, "offsets", torch.int32, (seqs + 1,))
        self.page_table, self.start, self.offsets = page_table, start, offsets
        self.tokens, self.max_new, self.max_len = int(tokens), int(max_new), int(max_len)
        self.struct = KVBatch._Struct(page_table.data_ptr(), start.data_ptr(), offsets.data_ptr(), seqs, stride,
                                      self.tokens, self.max_new, self.max_len)
        self.address = ctypes.addressof(self.struct)


def bl_kv_append(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, rope: Rope | None = None,
                 q: torch.Tensor | None = None, q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Writes the step's bf16 keys and values ``[tokens][heads][dim]`` into the cache, keys rotated on the way if
    there is a ``rope``; with it, ``q`` [tokens][q_heads][dim] is rotated too and returned (dense)."""
    shape = (batch.tokens, cache.heads, cache.dim)
    kp, kt, kh = _heads(k, "k", shape)
    vp, vt, vh = _heads(v, "v", shape)
    qp = qt = qh = q_heads = out = None
    if q is not None:
        if rope is None:
            raise ValueError("q is only rotated: it needs a rope")
        q_heads = q.shape[1]
        q_shape = (batch.tokens, q_heads, cache.dim)
        qp, qt, qh = _heads(q, "q", q_shape)
        if q_out is None:
            q_out = torch.empty(q_shape, dtype=torch.bfloat16, device=q.device)
        out = _dense(q_out, "q_out", torch.bfloat16, q_shape)
    _check("bl_kv_append", _lib.bl_kv_append(cache.address, batch.address, kp, kt, kh, vp, vt, vh,
                                             rope.address if rope is not None else None, qp, qt or 0, qh or 0,
                                             q_heads or 0, out, _stream(k.device)))
    return q_out if q is not None else None


def bl_kv_read(cache: KVCache, batch: KVBatch, k: torch.Tensor | None = None, v: torch.Tensor | None = None):
    """The batch's tokens as the cache holds them: bf16 k, v ``[tokens][heads][dim]``."""
    shape, dev = (batch.tokens, cache.heads, cache.dim), cache.k.device
    if k is None:
        k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if v is None:
        v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _check("bl_kv_read", _lib.bl_kv_read(cache.address, batch.address, _dense(k, "k", torch.bfloat16, shape),
                                         _dense(v, "v", torch.bfloat16, shape), _stream(dev)))
    return k, v


def bl_attention_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int) -> int:
    return int(_lib.bl_attention_workspace_bytes(cache.address, batch.address, q_heads))


def bl_attention(cache: KVCache, batch: KVBatch, q: torch.Tensor, scale: float | None = None, window: int = 0,
                 sinks: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the step's bf16 queries ``[tokens][q_heads][dim]`` over the cache (which holds the step's own
    tokens): bf16, dense.  ``scale`` is 1 / sqrt(dim) by default; ``window`` > 0 leaves the last ``window`` positions
    and the first ``sinks`` visible; ``lse`` (fp32 [tokens][q_heads]) takes the logarithms of the softmax sums."""
    q_heads = q.shape[1]
    shape = (batch.tokens, q_heads, cache.dim)
    qp, qt, qh = _heads(q, "q", shape)
    if scale is None:
        scale = cache.dim ** -0.5
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    if workspace is None:
        nbytes = _lib.bl_attention_workspace_bytes(cache.address, batch.address, q_heads)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    _check("bl_attention", _lib.bl_attention(cache.address, batch.address, qp, qt, qh, q_heads, scale, window, sinks,
                                             _dense(out, "out", torch.bfloat16, shape),
                                             _dense(lse, "lse", torch.float32, shape[:2]), workspace.data_ptr(), _bytes(workspace),
                                             _stream(q.device)))
    return out
