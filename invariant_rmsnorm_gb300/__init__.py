"""Python binding of the GB300 batch-invariant RMSNorm library (C ABI in
``include/rmsnorm.h``, ``layernorm.h`` and ``rope.h``).

Argument marshalling only: every function here takes torch tensors that the
caller allocated on a CUDA device, checks dtypes/shapes/devices, and passes raw
pointers, row strides and sizes to the ``extern "C"`` entry point of the same
name in ``_build/librmsnorm_gb300.so`` (LayerNorm and the rotary calls: through
``norm_call`` of ``include/slots.h``, one packed array in place of a conversion
an argument). All arithmetic runs in the library's
sm_103a kernels. If the library has not been built, ``load()`` raises; there is
no other implementation to fall back to.

Activations are bf16 ``[T, D]`` (bf16 or fp16 for the ``*_ex`` calls, which take
the format from ``x``) with unit column stride (any row stride that is a
multiple of 8 elements); weights and weight gradients fp32 ``[D]``;
inverse RMS fp32 ``[T]``. Work is enqueued on ``stream`` (default: the current
torch stream of the tensors' device).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "load", "lib_path", "RmsNormError", "workspace_bytes",
    "rmsnorm_fwd", "rmsnorm_bwd", "rmsnorm_residual_fwd", "rmsnorm_residual_bwd",
    "rmsnorm_gated_fwd", "rmsnorm_gated_bwd", "rmsnorm_dgamma_reduce",
    "rmsnorm_bwd_workspace_bytes", "rmsnorm_status_string", "rmsnorm_device_error",
    "rmsnorm_bwd_noalloc", "rmsnorm_fused_add_fwd", "rmsnorm_fused_add_bwd", "rmsnorm_bwd_recompute",
    "rmsnorm_gated_bwd_recompute", "rmsnorm_gated_hf_fwd", "EXPORTED_SYMBOLS",
    "rmsnorm_fwd_ex", "rmsnorm_bwd_ex", "rmsnorm_residual_fwd_ex", "rmsnorm_residual_bwd_ex",
    "rmsnorm_gated_fwd_ex", "rmsnorm_gated_bwd_ex", "rmsnorm_fused_add_fwd_ex", "rmsnorm_fused_add_bwd_ex",
    "rmsnorm_bwd_recompute_ex", "rmsnorm_gated_bwd_recompute_ex", "DTYPE_CODES", "GATE_CODES",
    "rmsnorm_residual_step_host", "rmsnorm_residual_step_host_work_bytes", "rmsnorm_selftest_wait_timeout",
    "DEVICE_ERR_WAIT_TIMEOUT", "rmsnorm_bwd_workspace_bytes_max",
    "rmsnorm_rope_fwd", "rmsnorm_rope_bwd", "rmsnorm_rope_bwd_workspace_bytes",
    "layernorm_fwd", "layernorm_bwd", "layernorm_bwd_workspace_bytes", "layernorm_bwd_workspace_bytes_max",
    "rope_fwd", "rope_bwd", "rope_frequencies", "LAYERNORM_SYMBOLS", "ROPE_SYMBOLS", "SLOTS_SYMBOLS", "ROPE_SCALINGS",
]

EXPORTED_SYMBOLS = (
    "rmsnorm_status_string", "rmsnorm_fwd", "rmsnorm_bwd_workspace_bytes", "rmsnorm_bwd",
    "rmsnorm_residual_fwd", "rmsnorm_residual_bwd", "rmsnorm_gated_fwd", "rmsnorm_gated_bwd",
    "rmsnorm_dgamma_reduce", "rmsnorm_device_error", "rmsnorm_bwd_noalloc",
    "rmsnorm_fused_add_fwd", "rmsnorm_fused_add_bwd", "rmsnorm_bwd_recompute", "rmsnorm_gated_bwd_recompute",
    "rmsnorm_gated_hf_fwd",
    "rmsnorm_fwd_ex", "rmsnorm_bwd_ex", "rmsnorm_residual_fwd_ex", "rmsnorm_residual_bwd_ex",
    "rmsnorm_gated_fwd_ex", "rmsnorm_gated_bwd_ex", "rmsnorm_fused_add_fwd_ex", "rmsnorm_fused_add_bwd_ex",
    "rmsnorm_bwd_recompute_ex", "rmsnorm_gated_bwd_recompute_ex",
    "rmsnorm_residual_step_host_work_bytes", "rmsnorm_residual_step_host", "rmsnorm_selftest_wait_timeout",
    "rmsnorm_bwd_workspace_bytes_max",
    "rmsnorm_rope_fwd", "rmsnorm_rope_bwd", "rmsnorm_rope_bwd_workspace_bytes",
)

# the entry points of include/layernorm.h and include/rope.h
LAYERNORM_SYMBOLS = ("layernorm_fwd", "layernorm_bwd", "layernorm_bwd_workspace_bytes",
                     "layernorm_bwd_workspace_bytes_max")
ROPE_SYMBOLS = ("rope_frequencies", "rope_fwd", "rope_bwd")
# of include/slots.h
SLOTS_SYMBOLS = ("norm_call",)

# RMSN_DEVICE_ERR_WAIT_TIMEOUT of include/rmsnorm.h: the flag a wait that ran out of time raises
DEVICE_ERR_WAIT_TIMEOUT = 1

# enum rmsn_dtype / enum rmsn_gate of include/rmsnorm.h
DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1}
GATE_CODES = {"silu": 0, "sigmoid": 1}

# enum rope_scaling of include/rope.h
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp_turns": 3, "ramp_index": 4}

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F = ctypes.c_float
_DBL = ctypes.c_double
_SZ = ctypes.c_size_t

_SIGS = {
    "rmsnorm_status_string": (ctypes.c_char_p, [_INT]),
    "rmsnorm_fwd": (_INT, [_P, _I64, _P, _P, _I64, _P, _I64, _I64, _F, _INT, _P]),
    "rmsnorm_bwd_workspace_bytes": (_SZ, [_I64, _I64]),
    "rmsnorm_bwd": (_INT, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _P, _SZ, _I64, _I64, _INT, _P]),
    "rmsnorm_residual_fwd": (_INT, [_P, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _F, _INT, _P]),
    "rmsnorm_residual_bwd": (_INT, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _SZ,
                                    _I64, _I64, _INT, _P]),
    "rmsnorm_gated_fwd": (_INT, [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _F, _INT, _P]),
    "rmsnorm_gated_hf_fwd": (_INT, [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _F, _INT, _P]),
    "rmsnorm_gated_bwd": (_INT, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P,
                                 _SZ, _I64, _I64, _INT, _P]),
    "rmsnorm_dgamma_reduce": (_INT, [_P, _SZ, _I64, _I64, _P, _P]),
    "rmsnorm_device_error": (_INT, [ctypes.POINTER(ctypes.c_uint), _INT]),
    "rmsnorm_bwd_noalloc": (_INT, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _I64, _INT, _P]),
    "rmsnorm_fused_add_fwd": (_INT, [_P, _I64, _P, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _F, _INT, _P]),
    "rmsnorm_fused_add_bwd": (_INT, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _SZ,
                                     _I64, _I64, _INT, _P]),
    "rmsnorm_bwd_recompute": (_INT, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _I64, _P, _SZ,
                                     _I64, _I64, _INT, _P]),
    "rmsnorm_gated_bwd_recompute": (_INT, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _I64,
                                           _P, _SZ, _I64, _I64, _INT, _P]),
}
_SIGS["rmsnorm_residual_step_host_work_bytes"] = (_SZ, [_I64, _I64, _I64])
_SIGS["rmsnorm_bwd_workspace_bytes_max"] = (_SZ, [_I64, _I64])
_SIGS["rmsnorm_selftest_wait_timeout"] = (_INT, [ctypes.c_ulonglong, _P, _P])
_SIGS["rmsnorm_residual_step_host"] = (_INT, [_P] * 9 + [_I64, _I64, _F, _INT, _INT, _I64, _P, _SZ, _P])
# Each *_ex call: the unsuffixed signature with `int dtype` (gated: `int gate, int dtype`) before the stream.
for _name in ("rmsnorm_fwd", "rmsnorm_bwd", "rmsnorm_residual_fwd", "rmsnorm_residual_bwd",
              "rmsnorm_fused_add_fwd", "rmsnorm_fused_add_bwd", "rmsnorm_gated_fwd", "rmsnorm_gated_bwd",
              "rmsnorm_bwd_recompute", "rmsnorm_gated_bwd_recompute"):
    _res, _args = _SIGS[_name]
    _extra = [_INT, _INT] if "gated" in _name else [_INT]
    _SIGS[_name + "_ex"] = (_res, _args[:-1] + _extra + [_P])
del _name, _res, _args, _extra

# A heads tensor is its pointer, token stride and head stride.
_HEADS = [_P, _I64, _I64]
_SIGS["layernorm_fwd"] = (_INT, [_P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _I64, _F, _INT, _INT, _P])
_SIGS["layernorm_bwd"] = (_INT, [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _P, _SZ, _I64, _I64, _INT, _INT,
                                 _P])
_SIGS["layernorm_bwd_workspace_bytes"] = (_SZ, [_I64, _I64])
_SIGS["layernorm_bwd_workspace_bytes_max"] = (_SZ, [_I64, _I64])
_SIGS["rope_frequencies"] = (_INT, [_I64, _DBL, _INT, _DBL, _DBL, _DBL, _DBL, _P])
_SIGS["rope_fwd"] = _SIGS["rope_bwd"] = (_INT, _HEADS * 2 + [_P, _P, _INT] + _HEADS * 2 + [_I64] * 5 +
                                         [_F, _INT, _INT, _P])
_SIGS["rmsnorm_rope_fwd"] = (_INT, _HEADS * 2 + [_P, _P, _P, _P, _INT] + _HEADS * 2 + [_P, _P] + [_I64] * 5 +
                             [_F, _INT, _F, _INT, _INT, _P])
_SIGS["rmsnorm_rope_bwd_workspace_bytes"] = (_SZ, [_I64] * 4)
_SIGS["rmsnorm_rope_bwd"] = (_INT, _HEADS * 4 + [_P, _P, _P, _P, _INT, _P, _P] + _HEADS * 2 + [_P, _P, _P, _SZ] +
                             [_I64] * 5 + [_F, _INT, _INT, _INT, _P])

# The entry points that are called with their arguments in an array (include/slots.h):
# enum norm_entry, the array's packing and its length.
_SIGS["norm_call"] = (_INT, [_INT, ctypes.c_char_p, _I64])
_SLOTS = {}
for _entry, _name in enumerate(("layernorm_fwd", "layernorm_bwd", "rope_fwd", "rope_bwd", "rmsnorm_rope_fwd",
                                "rmsnorm_rope_bwd")):
    _args = _SIGS[_name][1]
    _SLOTS[_name] = (_entry, struct.Struct("=" + "".join("d" if a is _F else "q" for a in _args)).pack, len(_args))
del _entry, _name, _args

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


class RmsNormError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {rmsnorm_status_string(status)} (status {status})")


def lib_path() -> str:
    return _build.lib_path()


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the shared library (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or lib_path()
            if not os.path.exists(p):
                raise RuntimeError(
                    f"CUDA library not built ({p} missing): run `python -c \"import __graft_entry__ as g; "
                    f"g.build()\"` first. There is no non-CUDA implementation.")
            lib = ctypes.CDLL(p)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _act(t: torch.Tensor, name: str, T: int, D: int, dtype: torch.dtype = torch.bfloat16) -> int:
    if t.dtype != dtype or not t.is_cuda or t.dim() != 2:
        raise TypeError(f"{name}: expected a 2-D {dtype} CUDA tensor, got {t.dtype} {t.device} {tuple(t.shape)}")
    if tuple(t.shape) != (T, D):
        raise ValueError(f"{name}: expected shape {(T, D)}, got {tuple(t.shape)}")
    if D > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: columns must be contiguous")
    return t.stride(0) if T > 1 else max(t.stride(0), D)


def _f32(t: torch.Tensor, name: str, n: int):
    if t.dtype != torch.float32 or not t.is_cuda or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise TypeError(f"{name}: expected a contiguous fp32 CUDA tensor of shape ({n},)")


def _stream(stream, dev) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    return ctypes.c_void_p(stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream))


def _check(fn: str, status: int):
    if status != 0:
        raise RmsNormError(fn, status)


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype not in DTYPE_CODES:
        raise TypeError(f"activations must be bf16 or fp16, got {x.dtype}")
    return DTYPE_CODES[x.dtype]


def _gate_code(gate: str) -> int:
    if gate not in GATE_CODES:
        raise ValueError(f"gate must be one of {sorted(GATE_CODES)}, got {gate!r}")
    return GATE_CODES[gate]


def _ws(ws: torch.Tensor):
    if not ws.is_cuda:
        raise TypeError("ws: expected a CUDA tensor")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


# --------------------------------------------------------------------------
# entry points (same names as the C ABI)
# --------------------------------------------------------------------------
def rmsnorm_status_string(status: int) -> str:
    return load().rmsnorm_status_string(int(status)).decode()


def rmsnorm_bwd_workspace_bytes(T: int, D: int) -> int:
    return int(load().rmsnorm_bwd_workspace_bytes(int(T), int(D)))


workspace_bytes = rmsnorm_bwd_workspace_bytes


def rmsnorm_bwd_workspace_bytes_max(T_max: int, D: int) -> int:
    """Bytes of one workspace that serves every T up to T_max (the per-T size is
    not monotone in T at some widths)."""
    return int(load().rmsnorm_bwd_workspace_bytes_max(int(T_max), int(D)))


def rmsnorm_fwd(x, w, y, rstd, eps: float = 1e-6, zero_centered_gamma: bool = False, stream=None):
    T, D = x.shape
    ldx, ldy = _act(x, "x", T, D), _act(y, "y", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_fwd", load().rmsnorm_fwd(_ptr(x), ldx, _ptr(w), _ptr(y), ldy, _ptr(rstd), T, D,
                                             float(eps), int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_residual_fwd(x, w, y, rstd, x_copy, eps: float = 1e-6, zero_centered_gamma: bool = False,
                         stream=None):
    T, D = x.shape
    ldx, ldy, ldc = _act(x, "x", T, D), _act(y, "y", T, D), _act(x_copy, "x_copy", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_residual_fwd", load().rmsnorm_residual_fwd(
        _ptr(x), ldx, _ptr(w), _ptr(y), ldy, _ptr(rstd), _ptr(x_copy), ldc, T, D, float(eps),
        int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_gated_fwd(x, z, w, y, rstd, eps: float = 1e-6, zero_centered_gamma: bool = True, stream=None):
    T, D = x.shape
    ldx, ldz, ldy = _act(x, "x", T, D), _act(z, "z", T, D), _act(y, "y", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_gated_fwd", load().rmsnorm_gated_fwd(
        _ptr(x), ldx, _ptr(z), ldz, _ptr(w), _ptr(y), ldy, _ptr(rstd), T, D, float(eps),
        int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_gated_hf_fwd(x, z, w, y, rstd, eps: float = 1e-6, zero_centered_gamma: bool = False, stream=None):
    """Gated forward in the HF convention (bf16 casts around the weight multiply)."""
    T, D = x.shape
    ldx, ldz, ldy = _act(x, "x", T, D), _act(z, "z", T, D), _act(y, "y", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_gated_hf_fwd", load().rmsnorm_gated_hf_fwd(
        _ptr(x), ldx, _ptr(z), ldz, _ptr(w), _ptr(y), ldy, _ptr(rstd), T, D, float(eps),
        int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_bwd(g, x, w, rstd, dx, dgamma, ws, zero_centered_gamma: bool = False, stream=None):
    """``dgamma`` may be None: pass 1 only (partials stay in ``ws``)."""
    T, D = x.shape
    ldg, ldx, lddx = _act(g, "g", T, D), _act(x, "x", T, D), _act(dx, "dx", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_bwd", load().rmsnorm_bwd(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(w), _ptr(rstd), _ptr(dx), lddx, _ptr(dgamma), wp, wb, T, D,
        int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_residual_bwd(g, x, w, rstd, g_res, dx, dgamma, ws, zero_centered_gamma: bool = False,
                         stream=None):
    """``g_res`` may be None (zero); ``dgamma`` may be None (pass 1 only)."""
    T, D = x.shape
    ldg, ldx, lddx = _act(g, "g", T, D), _act(x, "x", T, D), _act(dx, "dx", T, D)
    ldgr = _act(g_res, "g_res", T, D) if g_res is not None else D
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_residual_bwd", load().rmsnorm_residual_bwd(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(w), _ptr(rstd), _ptr(g_res), ldgr, _ptr(dx), lddx, _ptr(dgamma),
        wp, wb, T, D, int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_gated_bwd(g, x, z, w, rstd, dx, dz, dw, ws, zero_centered_gamma: bool = True, stream=None):
    """``dw`` may be None (pass 1 only)."""
    T, D = x.shape
    ldg, ldx, ldz = _act(g, "g", T, D), _act(x, "x", T, D), _act(z, "z", T, D)
    lddx, lddz = _act(dx, "dx", T, D), _act(dz, "dz", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dw is not None:
        _f32(dw, "dw", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_gated_bwd", load().rmsnorm_gated_bwd(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(z), ldz, _ptr(w), _ptr(rstd), _ptr(dx), lddx, _ptr(dz), lddz,
        _ptr(dw), wp, wb, T, D, int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_fused_add_fwd(x, res, w, y, rstd, res_out, eps: float = 1e-6, zero_centered_gamma: bool = False,
                          stream=None):
    """Norm of h = x + res (fp32); also writes bf16(h) to ``res_out``."""
    T, D = x.shape
    ldx, ldr, ldy, ldo = _act(x, "x", T, D), _act(res, "res", T, D), _act(y, "y", T, D), _act(res_out, "res_out", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_fused_add_fwd", load().rmsnorm_fused_add_fwd(
        _ptr(x), ldx, _ptr(res), ldr, _ptr(w), _ptr(y), ldy, _ptr(rstd), _ptr(res_out), ldo, T, D, float(eps),
        int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_fused_add_bwd(g, x, res, w, rstd, g_res, dh, dgamma, ws, zero_centered_gamma: bool = False,
                          stream=None):
    """Gradient of h = x + res (that of both x and res); ``g_res`` may be None."""
    T, D = x.shape
    ldg, ldx, ldr, ldd = _act(g, "g", T, D), _act(x, "x", T, D), _act(res, "res", T, D), _act(dh, "dh", T, D)
    ldgr = _act(g_res, "g_res", T, D) if g_res is not None else D
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_fused_add_bwd", load().rmsnorm_fused_add_bwd(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(res), ldr, _ptr(w), _ptr(rstd), _ptr(g_res), ldgr, _ptr(dh), ldd,
        _ptr(dgamma), wp, wb, T, D, int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_bwd_recompute(g, x, w, rstd, g_res, dx, dgamma, y, ws, zero_centered_gamma: bool = False,
                          stream=None):
    """rmsnorm_residual_bwd (``g_res`` may be None) that also writes the forward's y."""
    T, D = x.shape
    ldg, ldx, lddx, ldy = _act(g, "g", T, D), _act(x, "x", T, D), _act(dx, "dx", T, D), _act(y, "y", T, D)
    ldgr = _act(g_res, "g_res", T, D) if g_res is not None else D
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_bwd_recompute", load().rmsnorm_bwd_recompute(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(w), _ptr(rstd), _ptr(g_res), ldgr, _ptr(dx), lddx, _ptr(dgamma),
        _ptr(y), ldy, wp, wb, T, D, int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_gated_bwd_recompute(g, x, z, w, rstd, dx, dz, dw, y, ws, zero_centered_gamma: bool = True,
                                stream=None):
    """rmsnorm_gated_bwd that also writes the gated forward's y."""
    T, D = x.shape
    ldg, ldx, ldz = _act(g, "g", T, D), _act(x, "x", T, D), _act(z, "z", T, D)
    lddx, lddz, ldy = _act(dx, "dx", T, D), _act(dz, "dz", T, D), _act(y, "y", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dw is not None:
        _f32(dw, "dw", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_gated_bwd_recompute", load().rmsnorm_gated_bwd_recompute(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(z), ldz, _ptr(w), _ptr(rstd), _ptr(dx), lddx, _ptr(dz), lddz, _ptr(dw),
        _ptr(y), ldy, wp, wb, T, D, int(zero_centered_gamma), _stream(stream, x.device)))


# --------------------------------------------------------------------------
# activation dtype (bf16 / fp16, from x) and gate (silu / sigmoid) options
# --------------------------------------------------------------------------
def rmsnorm_fwd_ex(x, w, y, rstd, eps: float = 1e-6, zero_centered_gamma: bool = False, stream=None):
    T, D = x.shape
    dt = x.dtype
    ldx, ldy = _act(x, "x", T, D, dt), _act(y, "y", T, D, dt)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_fwd_ex", load().rmsnorm_fwd_ex(
        _ptr(x), ldx, _ptr(w), _ptr(y), ldy, _ptr(rstd), T, D, float(eps), int(zero_centered_gamma),
        _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_bwd_ex(g, x, w, rstd, dx, dgamma, ws, zero_centered_gamma: bool = False, stream=None):
    T, D = x.shape
    dt = x.dtype
    ldg, ldx, lddx = _act(g, "g", T, D, dt), _act(x, "x", T, D, dt), _act(dx, "dx", T, D, dt)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_bwd_ex", load().rmsnorm_bwd_ex(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(w), _ptr(rstd), _ptr(dx), lddx, _ptr(dgamma), wp, wb, T, D,
        int(zero_centered_gamma), _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_residual_fwd_ex(x, w, y, rstd, x_copy, eps: float = 1e-6, zero_centered_gamma: bool = False,
                            stream=None):
    T, D = x.shape
    dt = x.dtype
    ldx, ldy, ldc = _act(x, "x", T, D, dt), _act(y, "y", T, D, dt), _act(x_copy, "x_copy", T, D, dt)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_residual_fwd_ex", load().rmsnorm_residual_fwd_ex(
        _ptr(x), ldx, _ptr(w), _ptr(y), ldy, _ptr(rstd), _ptr(x_copy), ldc, T, D, float(eps),
        int(zero_centered_gamma), _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_residual_bwd_ex(g, x, w, rstd, g_res, dx, dgamma, ws, zero_centered_gamma: bool = False,
                            stream=None):
    T, D = x.shape
    dt = x.dtype
    ldg, ldx, lddx = _act(g, "g", T, D, dt), _act(x, "x", T, D, dt), _act(dx, "dx", T, D, dt)
    ldgr = _act(g_res, "g_res", T, D, dt) if g_res is not None else D
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_residual_bwd_ex", load().rmsnorm_residual_bwd_ex(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(w), _ptr(rstd), _ptr(g_res), ldgr, _ptr(dx), lddx, _ptr(dgamma),
        wp, wb, T, D, int(zero_centered_gamma), _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_gated_fwd_ex(x, z, w, y, rstd, eps: float = 1e-6, zero_centered_gamma: bool = True,
                         gate: str = "silu", stream=None):
    T, D = x.shape
    dt = x.dtype
    ldx, ldz, ldy = _act(x, "x", T, D, dt), _act(z, "z", T, D, dt), _act(y, "y", T, D, dt)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_gated_fwd_ex", load().rmsnorm_gated_fwd_ex(
        _ptr(x), ldx, _ptr(z), ldz, _ptr(w), _ptr(y), ldy, _ptr(rstd), T, D, float(eps),
        int(zero_centered_gamma), _gate_code(gate), _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_gated_bwd_ex(g, x, z, w, rstd, dx, dz, dw, ws, zero_centered_gamma: bool = True,
                         gate: str = "silu", stream=None):
    T, D = x.shape
    dt = x.dtype
    ldg, ldx, ldz = _act(g, "g", T, D, dt), _act(x, "x", T, D, dt), _act(z, "z", T, D, dt)
    lddx, lddz = _act(dx, "dx", T, D, dt), _act(dz, "dz", T, D, dt)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dw is not None:
        _f32(dw, "dw", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_gated_bwd_ex", load().rmsnorm_gated_bwd_ex(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(z), ldz, _ptr(w), _ptr(rstd), _ptr(dx), lddx, _ptr(dz), lddz,
        _ptr(dw), wp, wb, T, D, int(zero_centered_gamma), _gate_code(gate), _dtype_code(x),
        _stream(stream, x.device)))


def rmsnorm_fused_add_fwd_ex(x, res, w, y, rstd, res_out, eps: float = 1e-6, zero_centered_gamma: bool = False,
                             stream=None):
    T, D = x.shape
    dt = x.dtype
    ldx, ldr = _act(x, "x", T, D, dt), _act(res, "res", T, D, dt)
    ldy, ldo = _act(y, "y", T, D, dt), _act(res_out, "res_out", T, D, dt)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    _check("rmsnorm_fused_add_fwd_ex", load().rmsnorm_fused_add_fwd_ex(
        _ptr(x), ldx, _ptr(res), ldr, _ptr(w), _ptr(y), ldy, _ptr(rstd), _ptr(res_out), ldo, T, D, float(eps),
        int(zero_centered_gamma), _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_fused_add_bwd_ex(g, x, res, w, rstd, g_res, dh, dgamma, ws, zero_centered_gamma: bool = False,
                             stream=None):
    T, D = x.shape
    dt = x.dtype
    ldg, ldx = _act(g, "g", T, D, dt), _act(x, "x", T, D, dt)
    ldr, ldd = _act(res, "res", T, D, dt), _act(dh, "dh", T, D, dt)
    ldgr = _act(g_res, "g_res", T, D, dt) if g_res is not None else D
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_fused_add_bwd_ex", load().rmsnorm_fused_add_bwd_ex(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(res), ldr, _ptr(w), _ptr(rstd), _ptr(g_res), ldgr, _ptr(dh), ldd,
        _ptr(dgamma), wp, wb, T, D, int(zero_centered_gamma), _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_bwd_recompute_ex(g, x, w, rstd, g_res, dx, dgamma, y, ws, zero_centered_gamma: bool = False,
                             stream=None):
    T, D = x.shape
    dt = x.dtype
    ldg, ldx, lddx, ldy = _act(g, "g", T, D, dt), _act(x, "x", T, D, dt), _act(dx, "dx", T, D, dt), _act(y, "y", T, D, dt)
    ldgr = _act(g_res, "g_res", T, D, dt) if g_res is not None else D
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_bwd_recompute_ex", load().rmsnorm_bwd_recompute_ex(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(w), _ptr(rstd), _ptr(g_res), ldgr, _ptr(dx), lddx, _ptr(dgamma),
        _ptr(y), ldy, wp, wb, T, D, int(zero_centered_gamma), _dtype_code(x), _stream(stream, x.device)))


def rmsnorm_gated_bwd_recompute_ex(g, x, z, w, rstd, dx, dz, dw, y, ws, zero_centered_gamma: bool = True,
                                   gate: str = "silu", stream=None):
    T, D = x.shape
    dt = x.dtype
    ldg, ldx, ldz = _act(g, "g", T, D, dt), _act(x, "x", T, D, dt), _act(z, "z", T, D, dt)
    lddx, lddz, ldy = _act(dx, "dx", T, D, dt), _act(dz, "dz", T, D, dt), _act(y, "y", T, D, dt)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dw is not None:
        _f32(dw, "dw", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_gated_bwd_recompute_ex", load().rmsnorm_gated_bwd_recompute_ex(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(z), ldz, _ptr(w), _ptr(rstd), _ptr(dx), lddx, _ptr(dz), lddz, _ptr(dw),
        _ptr(y), ldy, wp, wb, T, D, int(zero_centered_gamma), _gate_code(gate), _dtype_code(x),
        _stream(stream, x.device)))


# --------------------------------------------------------------------------
# LayerNorm, rotary positions, and the head RMSNorm fused with them
# --------------------------------------------------------------------------
# The calls of this section are short enough on the GPU for their checks to count,
# so these are plain functions of a tensor and the device's index, the passing case
# first, and each returns what the entry point takes.
_F32, _F64 = torch.float32, torch.float64


def _index_and_code(x: torch.Tensor, name: str):
    """The device of a call (its first tensor's) and the activation format's code."""
    code = DTYPE_CODES.get(x.dtype)
    if code is None or not x.is_cuda:
        raise TypeError(f"{name}: expected a bf16 or fp16 CUDA tensor, got {x.dtype} {x.device}")
    return x.get_device(), code


def _rows(t, name: str, shape, dtype, index: int):
    """Pointer and row stride of an activation matrix."""
    if t.dtype is dtype and t.get_device() == index and t.shape == shape:
        ld, one = t.stride()
        if one == 1 or shape[1] <= 1:
            return t.data_ptr(), ld if shape[0] > 1 else shape[1]  # a stride that is never taken may be anything
        raise ValueError(f"{name}: columns must be contiguous")
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 2:
        raise TypeError(f"{name}: expected a 2-D {dtype} tensor on cuda:{index}, got {t.dtype} {t.device} {tuple(t.shape)}")
    raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _heads(t, name: str, shape, dtype, index: int):
    """Pointer, token stride and head stride of [T, heads, D] (None: of no heads)."""
    if t is None:
        if shape[1] == 0:
            return 0, 0, 0
        raise TypeError(f"{name}: expected a tensor of shape {shape}")
    if t.dtype is dtype and t.get_device() == index and t.shape == shape:
        token, head, one = t.stride()
        if one == 1 or shape[2] <= 1:
            # a stride that is never taken may be anything
            return t.data_ptr(), token if shape[0] > 1 else 0, head if shape[1] > 1 else 0
        raise ValueError(f"{name}: the values of a head must be contiguous")
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 3:
        raise TypeError(f"{name}: expected a 3-D {dtype} tensor on cuda:{index}, got {t.dtype} {t.device} {tuple(t.shape)}")
    raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")


def _vec(t, name: str, shape, index: int, dtype: torch.dtype = _F32):
    """Pointer of a contiguous tensor of fp32 (or ``dtype``) values."""
    if t is not None and t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise TypeError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}" +
                    ("" if t is None else f", got {t.dtype} {t.device} {tuple(t.shape)}"))


def _bytes_of(ws, index: int):
    if ws.get_device() != index or not ws.is_contiguous():
        raise TypeError(f"ws: expected a contiguous tensor on cuda:{index}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _positions(t, T: int, index: int):
    """Pointer and enum rope_pos_dtype (None: 0, 1, 2, ...)."""
    if t is None:
        return 0, 1
    if t.dtype is torch.int64:
        return _vec(t, "positions", (T,), index, torch.int64), 1
    if t.dtype is torch.int32:
        return _vec(t, "positions", (T,), index, torch.int32), 0
    raise TypeError(f"positions: expected int32 or int64, got {t.dtype}")


# The current stream's handle and the current device without the objects around
# them, where torch has these (as of 2.x); the public calls otherwise.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _handle(stream, index: int) -> int:
    if stream is None:
        return _raw_stream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _call(name: str, index: int, stream, *args):
    """The entry point ``name`` on ``stream``, with the tensors' device current (a null pointer is 0)."""
    entry, pack, n = _SLOTS[name]
    slots = pack(*args, _handle(stream, index))
    fn = (_lib or load()).norm_call
    if _device_now() == index:
        st = fn(entry, slots, n)
    else:
        with torch.cuda.device(index):
            st = fn(entry, slots, n)
    if st != 0:
        raise RmsNormError(name, st)


def layernorm_fwd(x, w, b, y, mean, rstd, eps: float = 1e-5, zero_centered_gamma: bool = False, stream=None):
    """``y = (x - mean) * rstd * w_eff + b`` by rows; writes ``y``, ``mean``, ``rstd``. ``b`` may be None.
    The activation format (bf16 or fp16) is ``x``'s."""
    i, code = _index_and_code(x, "x")
    dt, shape = x.dtype, x.shape
    if len(shape) != 2:
        raise TypeError(f"x: expected a 2-D tensor [T, D], got {tuple(shape)}")
    T, D = shape
    xp, ldx = _rows(x, "x", shape, dt, i)
    yp, ldy = _rows(y, "y", shape, dt, i)
    _call("layernorm_fwd", i, stream, xp, ldx, _vec(w, "w", (D,), i), 0 if b is None else _vec(b, "b", (D,), i), yp, ldy,
          _vec(mean, "mean", (T,), i), _vec(rstd, "rstd", (T,), i), T, D, eps, 1 if zero_centered_gamma else 0, code)


def layernorm_bwd_workspace_bytes(T: int, D: int) -> int:
    return int(load().layernorm_bwd_workspace_bytes(int(T), int(D)))


def layernorm_bwd_workspace_bytes_max(T_max: int, D: int) -> int:
    """Bytes of one workspace that serves every T up to T_max."""
    return int(load().layernorm_bwd_workspace_bytes_max(int(T_max), int(D)))


def layernorm_bwd(g, x, w, mean, rstd, dx, dw, db, ws, zero_centered_gamma: bool = False, stream=None):
    """Writes ``dx``, ``dw`` and, unless it is None, ``db``. ``ws`` is a workspace of
    ``layernorm_bwd_workspace_bytes(T, D)`` bytes."""
    i, code = _index_and_code(x, "x")
    dt, shape = x.dtype, x.shape
    if len(shape) != 2:
        raise TypeError(f"x: expected a 2-D tensor [T, D], got {tuple(shape)}")
    T, D = shape
    gp, ldg = _rows(g, "g", shape, dt, i)
    xp, ldx = _rows(x, "x", shape, dt, i)
    dp, ldd = _rows(dx, "dx", shape, dt, i)
    wp, wb = _bytes_of(ws, i)
    _call("layernorm_bwd", i, stream, gp, ldg, xp, ldx, _vec(w, "w", (D,), i), _vec(mean, "mean", (T,), i),
          _vec(rstd, "rstd", (T,), i), dp, ldd, _vec(dw, "dw", (D,), i), 0 if db is None else _vec(db, "db", (D,), i), wp,
          wb, T, D, 1 if zero_centered_gamma else 0, code)


def rope_frequencies(R: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0, low: float = 1.0,
                     high: float = 32.0, length: float = 0.0) -> torch.Tensor:
    """The R/2 rotary frequencies (radians a position) as a float64 CPU tensor: ``theta ** (-2 i / R)``,
    scaled for contexts longer than those of training (the scalings of include/rope.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    out = torch.empty(max(int(R), 0) // 2, dtype=torch.float64)
    _check("rope_frequencies", load().rope_frequencies(int(R), float(theta), ROPE_SCALINGS[scaling], float(factor),
                                                       float(low), float(high), float(length), _ptr(out)))
    return out


def _q_k(q, k, inv_freq):
    """Shapes of q and k and the number of frequencies."""
    shape = q.shape
    if len(shape) != 3:
        raise TypeError(f"q: expected a 3-D tensor [T, heads, D], got {tuple(shape)}")
    if inv_freq.dim() != 1:
        raise TypeError(f"inv_freq: expected a 1-D tensor, got {tuple(inv_freq.shape)}")
    T, _, D = shape
    if k is None:
        return shape, (T, 0, D), inv_freq.shape[0]
    if k.dim() != 3:
        raise TypeError(f"k: expected a 3-D tensor [T, heads, D], got {tuple(k.shape)}")
    return shape, (T, k.shape[1], D), inv_freq.shape[0]


def _rope(name, q, k, inv_freq, q_out, k_out, positions, scale, interleaved, stream):
    i, code = _index_and_code(q, "q")
    dt = q.dtype
    sq, sk, n = _q_k(q, k, inv_freq)
    T, Hq, D = sq
    _call(name, i, stream, *_heads(q, "q", sq, dt, i), *_heads(k, "k", sk, dt, i), _vec(inv_freq, "inv_freq", (n,), i, _F64),
          *_positions(positions, T, i), *_heads(q_out, "q_out", sq, dt, i), *_heads(k_out, "k_out", sk, dt, i), T, Hq, sk[1],
          D, 2 * n, scale, 1 if interleaved else 0, code)


def rope_fwd(q, k, inv_freq, q_out, k_out, positions=None, scale: float = 1.0, interleaved: bool = False, stream=None):
    """Rotary positions of ``q`` [T, Hq, D] and ``k`` [T, Hk, D] (None: q alone): the first
    ``2 * len(inv_freq)`` values of each head in pairs (halves, or neighbours if ``interleaved``), turned by
    ``positions * inv_freq`` (float64 frequencies; positions None: 0, 1, 2, ...) and scaled by ``scale``.
    ``q_out`` may be ``q`` and ``k_out`` may be ``k``."""
    _rope("rope_fwd", q, k, inv_freq, q_out, k_out, positions, scale, interleaved, stream)


def rope_bwd(gq, gk, inv_freq, dq, dk, positions=None, scale: float = 1.0, interleaved: bool = False, stream=None):
    """Gradients of rope_fwd's inputs from those of its outputs (``dq`` may be ``gq``, ``dk`` may be ``gk``)."""
    _rope("rope_bwd", gq, gk, inv_freq, dq, dk, positions, scale, interleaved, stream)


def rmsnorm_rope_fwd(q, k, wq, wk, inv_freq, q_out, k_out, rstd_q, rstd_k, positions=None, scale: float = 1.0,
                     interleaved: bool = False, eps: float = 1e-6, zero_centered_gamma: bool = False, stream=None):
    """RMSNorm of every head of ``q`` (weight ``wq`` [D]) and of ``k`` (``wk``), then their rotary positions as
    in ``rope_fwd``, in one pass; writes ``q_out``, ``k_out`` and the inverse RMS of every head, ``rstd_q`` [T, Hq]
    and ``rstd_k`` [T, Hk]. ``k``, ``wk``, ``k_out`` and ``rstd_k`` may be None together."""
    i, code = _index_and_code(q, "q")
    dt = q.dtype
    sq, sk, n = _q_k(q, k, inv_freq)
    T, Hq, D = sq
    Hk = sk[1]
    _call("rmsnorm_rope_fwd", i, stream, *_heads(q, "q", sq, dt, i), *_heads(k, "k", sk, dt, i), _vec(wq, "wq", (D,), i),
          _vec(wk, "wk", (D,), i) if Hk else 0, _vec(inv_freq, "inv_freq", (n,), i, _F64), *_positions(positions, T, i),
          *_heads(q_out, "q_out", sq, dt, i), *_heads(k_out, "k_out", sk, dt, i), _vec(rstd_q, "rstd_q", (T, Hq), i),
          _vec(rstd_k, "rstd_k", (T, Hk), i) if Hk else 0, T, Hq, Hk, D, 2 * n, scale, 1 if interleaved else 0, eps,
          1 if zero_centered_gamma else 0, code)


def rmsnorm_rope_bwd_workspace_bytes(T: int, Hq: int, Hk: int, D: int) -> int:
    return int(load().rmsnorm_rope_bwd_workspace_bytes(int(T), int(Hq), int(Hk), int(D)))


def rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, inv_freq, rstd_q, rstd_k, dq, dk, dwq, dwk, ws, positions=None,
                     scale: float = 1.0, interleaved: bool = False, zero_centered_gamma: bool = False, stream=None):
    """Gradients of rmsnorm_rope_fwd: ``dq``, ``dk`` (which may be ``gq``, ``gk``) and the weights' ``dwq``, ``dwk``.
    ``ws`` is a workspace of ``rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D)`` bytes."""
    i, code = _index_and_code(q, "q")
    dt = q.dtype
    sq, sk, n = _q_k(q, k, inv_freq)
    T, Hq, D = sq
    Hk = sk[1]
    wp, wb = _bytes_of(ws, i)
    _call("rmsnorm_rope_bwd", i, stream, *_heads(gq, "gq", sq, dt, i), *_heads(gk, "gk", sk, dt, i),
          *_heads(q, "q", sq, dt, i), *_heads(k, "k", sk, dt, i), _vec(wq, "wq", (D,), i),
          _vec(wk, "wk", (D,), i) if Hk else 0, _vec(inv_freq, "inv_freq", (n,), i, _F64), *_positions(positions, T, i),
          _vec(rstd_q, "rstd_q", (T, Hq), i), _vec(rstd_k, "rstd_k", (T, Hk), i) if Hk else 0,
          *_heads(dq, "dq", sq, dt, i), *_heads(dk, "dk", sk, dt, i), _vec(dwq, "dwq", (D,), i),
          _vec(dwk, "dwk", (D,), i) if Hk else 0, wp, wb, T, Hq, Hk, D, 2 * n, scale, 1 if interleaved else 0,
          1 if zero_centered_gamma else 0, code)


def rmsnorm_dgamma_reduce(ws, T: int, D: int, dgamma, stream=None):
    _f32(dgamma, "dgamma", D)
    wp, wb = _ws(ws)
    _check("rmsnorm_dgamma_reduce", load().rmsnorm_dgamma_reduce(
        wp, wb, int(T), int(D), _ptr(dgamma), _stream(stream, dgamma.device)))


def rmsnorm_bwd_noalloc(g, x, w, rstd, dx, dgamma, zero_centered_gamma: bool = False, stream=None):
    """Backward for callers that cannot allocate device memory: the library's own
    fixed scratch array replaces the workspace (see include/rmsnorm.h)."""
    T, D = x.shape
    ldg, ldx, lddx = _act(g, "g", T, D), _act(x, "x", T, D), _act(dx, "dx", T, D)
    _f32(w, "w", D)
    _f32(rstd, "rstd", T)
    if dgamma is not None:
        _f32(dgamma, "dgamma", D)
    _check("rmsnorm_bwd_noalloc", load().rmsnorm_bwd_noalloc(
        _ptr(g), ldg, _ptr(x), ldx, _ptr(w), _ptr(rstd), _ptr(dx), lddx, _ptr(dgamma), T, D,
        int(zero_centered_gamma), _stream(stream, x.device)))


def rmsnorm_device_error(clear: bool = True) -> int:
    """Device-side error flags since the last clear (0 = none). Synchronises."""
    flags = ctypes.c_uint(0)
    _check("rmsnorm_device_error", load().rmsnorm_device_error(ctypes.byref(flags), int(clear)))
    return int(flags.value)


def _host(t: torch.Tensor, name: str, shape, dtype: torch.dtype):
    if t.dtype != dtype or t.is_cuda or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous host {dtype} tensor of shape {tuple(shape)}, got "
                        f"{t.dtype} {t.device} {tuple(t.shape)}")


def rmsnorm_residual_step_host_work_bytes(T: int, D: int, slab_rows: int = 0) -> int:
    return int(load().rmsnorm_residual_step_host_work_bytes(int(T), int(D), int(slab_rows)))


def rmsnorm_residual_step_host(x, g, g_res, w, y, x_copy, rstd, dx, dgamma, work, eps: float = 1e-6,
                               zero_centered_gamma: bool = False, slab_rows: int = 0, stream=None):
    """rmsnorm_residual forward + backward on HOST tensors (pinned for overlap):
    one call copies the inputs in, runs both kernels and copies every output
    back, pipelined in row slabs inside the library. ``work`` is a CUDA byte
    buffer of ``rmsnorm_residual_step_host_work_bytes(T, D, slab_rows)`` bytes;
    the host tensors must not be touched until ``stream`` has completed."""
    T, D = x.shape
    dt = x.dtype
    for t, n in ((x, "x"), (g, "g"), (y, "y"), (x_copy, "x_copy"), (dx, "dx")):
        _host(t, n, (T, D), dt)
    if g_res is not None:
        _host(g_res, "g_res", (T, D), dt)
    _host(w, "w", (D,), torch.float32)
    _host(dgamma, "dgamma", (D,), torch.float32)
    _host(rstd, "rstd", (T,), torch.float32)
    wp, wb = _ws(work)
    _check("rmsnorm_residual_step_host", load().rmsnorm_residual_step_host(
        _ptr(x), _ptr(g), _ptr(g_res), _ptr(w), _ptr(y), _ptr(x_copy), _ptr(rstd), _ptr(dx), _ptr(dgamma),
        T, D, float(eps), int(zero_centered_gamma), _dtype_code(x), int(slab_rows), wp, wb,
        _stream(stream, work.device)))


def rmsnorm_selftest_wait_timeout(limit_ns: int, waited_ns: Optional[torch.Tensor] = None, device=None, stream=None):
    """Runs the bounded-wait error path on purpose: one thread waits, with the
    kernels' own wait and a limit of ``limit_ns``, on a barrier nothing completes,
    then raises DEVICE_ERR_WAIT_TIMEOUT (read it with rmsnorm_device_error). If
    ``waited_ns`` (a CUDA int64 tensor of one element) is given, the time the wait
    took is written there."""
    if waited_ns is not None and (not waited_ns.is_cuda or waited_ns.dtype != torch.int64 or waited_ns.numel() != 1):
        raise TypeError("waited_ns: expected a one-element int64 CUDA tensor")
    dev = waited_ns.device if waited_ns is not None else (device or torch.device("cuda", torch.cuda.current_device()))
    _check("rmsnorm_selftest_wait_timeout", load().rmsnorm_selftest_wait_timeout(
        ctypes.c_ulonglong(int(limit_ns)), _ptr(waited_ns), _stream(stream, dev)))
