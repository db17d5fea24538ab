"""What a draft layer in 8 bits is made of: argument marshalling over eagle_rms_norm, eagle_quantize_rows and
eagle_linear of the C ABI (include/eagle_tree.h has the formulas).

An 8-bit row is e4m3 codes and one fp32 scale.  ``quantize_rows`` makes such rows of bf16 ones (weights once,
activations as they come), ``rms_norm`` ends in them, and ``linear`` multiplies them and applies scales, bias,
activation and residual on the accumulator.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import EAGLE_BF16, EAGLE_E4M3, EAGLE_F32, check
from .kv4 import _AS_IS

_BF16, _E4M3, _F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
_ACTS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "swiglu": 3}
_TICKETS = 4096  # bytes at the start of a workspace that are zero between calls


def _rows(t, name, dtype, index, shape=None):
    """Elements between the rows of a [rows][cols] matrix on the device, its last axis packed."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a matrix" + ("" if shape is None else f" of shape {tuple(shape)}"))
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: a row's elements must be packed")
    if rows > 1:
        if t.stride(0) < cols:
            raise ValueError(f"{name}: rows must not overlap")
        return t.stride(0)
    size = 16 // t.element_size()
    return (cols + size - 1) // size * size  # of one row: whatever the stride


def _vector(t, name, dtype, index, n):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}")
    return t.data_ptr()


def _index(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _on(index, stream):
    """Makes the operands' device current, and `stream` where one is given, so that what is allocated
    belongs to the stream that uses it."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the operands on cuda:{index}")
        return torch.cuda.stream(stream)
    return _AS_IS if torch.cuda.current_device() == index else torch.cuda.device(index)


def _raw(index, stream):
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _new_rows(like, rows, cols, dtype, step):
    """A [rows][cols] matrix whose rows start a multiple of `step` elements apart."""
    ld = (cols + step - 1) // step * step
    t = torch.empty((rows, ld), dtype=dtype, device=like.device)
    return t if ld == cols else t[:, :cols]


def quantize_rows(x, stream=None):
    """The rows of x [rows][cols] bf16 as 8-bit rows: (codes [rows][cols] float8_e4m3fn, scale [rows] fp32),
    codes times scale standing for x."""
    lib, index = _lib.load(), _index(x, "x")
    ldx = _rows(x, "x", _BF16, index)
    rows, cols = x.shape
    with _on(index, stream):
        y = _new_rows(x, rows, cols, _E4M3, 16)
        scale = torch.empty(rows, dtype=_F32, device=x.device)
        check(lib.eagle_quantize_rows(x.data_ptr(), ldx, rows, cols, y.data_ptr(), _rows(y, "y", _E4M3, index),
                                      scale.data_ptr(), _raw(index, stream)), "eagle_quantize_rows")
    return y, scale


def rms_norm(x, weight, eps: float = 1e-6, residual=None, dtype=torch.bfloat16, stream=None):
    """y = weight h / sqrt(mean(h^2) + eps) over the rows of h = x + residual (or x).  x and residual
    [rows][cols] bf16, weight [cols] bf16.  Returns (y, scale, h): y in bf16 (scale None), or with
    dtype=torch.float8_e4m3fn as codes with a scale [rows] fp32; h in bf16 where there is a residual, else
    None."""
    lib, index = _lib.load(), _index(x, "x")
    ldx = _rows(x, "x", _BF16, index)
    rows, cols = x.shape
    p_w = _vector(weight, "weight", _BF16, index, cols)
    if dtype is not _BF16 and dtype is not _E4M3:
        raise TypeError(f"rms_norm gives torch.bfloat16 or torch.float8_e4m3fn, not {dtype}")
    fp8 = dtype is _E4M3
    p_res, ldr, lds, p_sum, p_scale = None, 0, 0, None, None
    if residual is not None:
        ldr, p_res = _rows(residual, "residual", _BF16, index, x.shape), residual.data_ptr()
    with _on(index, stream):
        y = _new_rows(x, rows, cols, dtype, 16 if fp8 else 8)
        scale = total = None
        if fp8:
            scale = torch.empty(rows, dtype=_F32, device=x.device)
            p_scale = scale.data_ptr()
        if residual is not None:
            total = _new_rows(x, rows, cols, _BF16, 8)
            lds, p_sum = _rows(total, "h", _BF16, index), total.data_ptr()
        check(lib.eagle_rms_norm(x.data_ptr(), ldx, p_res, ldr, p_w, eps, rows, cols, p_sum, lds,
                                 EAGLE_E4M3 if fp8 else EAGLE_BF16, y.data_ptr(), _rows(y, "y", dtype, index), p_scale,
                                 _raw(index, stream)), "eagle_rms_norm")
    return y, scale, total


def linear_workspace(w, rows: int, stream=None):
    """Scratch for ``linear`` calls of up to `rows` rows on w's device, one call at a time."""
    lib, index = _lib.load(), _index(w, "w")
    with _on(index, stream):
        nbytes = lib.eagle_linear_epilogue_workspace_bytes(max(rows, 1))
        if nbytes == 0:
            raise ValueError(f"unusable number of rows ({rows})")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
        ws[:_TICKETS].zero_()
    return ws


def linear(w, x, bias=None, act=None, residual=None, w_scale=None, x_scale=None, dtype=torch.bfloat16, out=None,
           workspace=None, stream=None):
    """y = act(w_scale x_scale (x w^T) + bias) + residual.  w [features][k] and x [rows][k] are bf16, or
    8-bit rows (float8_e4m3fn) with w_scale [features] and x_scale [rows] fp32; bias [features] bf16; act None,
    "silu", "gelu" or "swiglu" (w: gate rows, then as many up rows; y = silu(gate) up); residual [rows][out]
    bf16.  Returns y [rows][out] of dtype (bf16 or fp32), or fills out, which may be the residual.  workspace:
    one of ``linear_workspace`` instead of a fresh one; calls that may overlap need one each."""
    lib, index = _lib.load(), _index(w, "w")
    kind = w.dtype
    if kind is not _BF16 and kind is not _E4M3:
        raise TypeError(f"w must be torch.bfloat16 or torch.float8_e4m3fn, got {kind}")
    if act not in _ACTS:
        raise ValueError(f"act must be one of None, 'silu', 'gelu', 'swiglu', got {act!r}")
    code = _ACTS[act]
    ldw, ldx = _rows(w, "w", kind, index), _rows(x, "x", kind, index)
    features, k = w.shape
    rows = x.shape[0]
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, w {k}")
    if code == 3 and features % 2:
        raise ValueError("swiglu needs as many up rows of w as gate rows")
    width = features // 2 if code == 3 else features
    fp8 = kind is _E4M3
    if fp8 != (w_scale is not None) or fp8 != (x_scale is not None):
        raise ValueError("8-bit operands have w_scale and x_scale, bf16 ones none")
    p_ws, p_xs = (_vector(w_scale, "w_scale", _F32, index, features), _vector(x_scale, "x_scale", _F32, index, rows)) if fp8 \
        else (None, None)
    p_bias = None if bias is None else _vector(bias, "bias", _BF16, index, features)
    p_res, ldr = None, 0
    if residual is not None:
        ldr, p_res = _rows(residual, "residual", _BF16, index, (rows, width)), residual.data_ptr()
    if out is not None:
        dtype = out.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"linear gives torch.bfloat16 or torch.float32, not {dtype}")
    with _on(index, stream):
        if out is None:
            out = _new_rows(x, rows, width, dtype, 8 if dtype is _BF16 else 4)
        ldy = _rows(out, "out", dtype, index, (rows, width))
        if workspace is None:
            workspace = linear_workspace(w, rows)
        elif workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
        args = _lib.LinearArgs(rows, width, k, EAGLE_E4M3 if fp8 else EAGLE_BF16, EAGLE_BF16 if dtype is _BF16 else EAGLE_F32,
                               code, w.data_ptr(), x.data_ptr(), ldw, ldx, p_ws, p_xs, p_bias, p_res, ldr, out.data_ptr(), ldy)
        check(lib.eagle_linear(ctypes.byref(args), workspace.data_ptr(), workspace.numel(), None, _raw(index, stream)),
              "eagle_linear")
    return out
