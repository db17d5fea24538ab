"""What a draft layer in 8 bits is made of: argument marshalling over eagle_rms_norm, eagle_quantize_rows and
eagle_linear of the C ABI (include/eagle_tree.h has the formulas).

An 8-bit row is e4m3 codes and one fp32 scale.  ``quantize_rows`` makes such rows of bf16 ones (weights once,
activations as they come), ``rms_norm`` ends in them, and ``linear`` multiplies them and applies scales, bias,
activation and residual on the accumulator.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import EAGLE_BF16, EAGLE_E4M3, EAGLE_F32, check, short
from .engine import _need

_BF16, _E4M3, _F32, _U8 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.uint8
_ACTS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "swiglu": 3}
_CODES = {torch.bfloat16: EAGLE_BF16, torch.float8_e4m3fn: EAGLE_E4M3, torch.float32: EAGLE_F32}
_AS_IS = contextlib.nullcontext()
_TICKETS = 4096  # bytes at the start of a workspace that are zero between calls


def _rows(t, name, dtype, index):
    """(rows, cols, elements between rows) of a matrix on device `index` whose rows are packed."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: a row's elements must be packed")
    if rows < 2:
        return rows, cols, (cols + 15) // 16 * 16  # whatever the strides of sizes of 1
    if ld < cols:
        raise ValueError(f"{name}: rows must not overlap")
    return rows, cols, ld


def _vector(t, name, dtype, index, n):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}")
    return t.data_ptr()


def _device(t, name):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _elsewhere(index, stream):
    """None where the operands' device is current and no stream is given; else a context in which they are,
    so that what is allocated belongs to the stream that uses it."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the operands on cuda:{index}")
        return torch.cuda.stream(stream)
    return None if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


_stream = torch._C._cuda_getCurrentRawStream


def _new_rows(like, rows, cols, dtype, step):
    """A [rows][cols] matrix whose rows start a multiple of `step` elements apart, and that multiple."""
    ld = (cols + step - 1) // step * step
    if ld == cols:
        return torch.empty((rows, cols), dtype=dtype, device=like.device), ld
    return torch.empty_strided((rows, cols), (ld, 1), dtype=dtype, device=like.device), ld


def quantize_rows(x, stream=None):
    """The rows of x [rows][cols] bf16 as 8-bit rows: (codes [rows][cols] float8_e4m3fn, scale [rows] fp32),
    codes times scale standing for x."""
    if stream is None:
        made = short.quantize_rows(x)
        if made is not NotImplemented:
            return made
    index = _device(x, "x")
    rows, cols, ldx = _rows(x, "x", _BF16, index)
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return quantize_rows(x)
    y, ldy = _new_rows(x, rows, cols, _E4M3, 16)
    scale = torch.empty(rows, dtype=_F32, device=x.device)
    check(_lib.load().eagle_quantize_rows(x.data_ptr(), ldx, rows, cols, y.data_ptr(), ldy, scale.data_ptr(), _stream(index)),
          "eagle_quantize_rows")
    return y, scale


def rms_norm(x, weight, eps: float = 1e-6, residual=None, dtype=torch.bfloat16, stream=None):
    """y = weight h / sqrt(mean(h^2) + eps) over the rows of h = x + residual (or x).  x and residual
    [rows][cols] bf16, weight [cols] bf16.  Returns (y, scale, h): y in bf16 (scale None), or with
    dtype=torch.float8_e4m3fn as codes with a scale [rows] fp32; h in bf16 where there is a residual, else
    None."""
    if stream is None and (dtype is _E4M3 or dtype is _BF16):
        made = short.rms_norm(x, weight, eps, residual, dtype is _E4M3)
        if made is not NotImplemented:
            return made
    index = _device(x, "x")
    rows, cols, ldx = _rows(x, "x", _BF16, index)
    p_w = _vector(weight, "weight", _BF16, index, cols)
    if dtype is not _BF16 and dtype is not _E4M3:
        raise TypeError(f"rms_norm gives torch.bfloat16 or torch.float8_e4m3fn, not {dtype}")
    p_res, ldr, lds, p_sum, p_scale, scale, total = None, 0, 0, None, None, None, None
    if residual is not None:
        r_rows, r_cols, ldr = _rows(residual, "residual", _BF16, index)
        if r_rows != rows or r_cols != cols:
            raise ValueError(f"residual must be [{rows}][{cols}]")
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return rms_norm(x, weight, eps, residual, dtype)
    if residual is not None:
        p_res = residual.data_ptr()
        total, lds = _new_rows(x, rows, cols, _BF16, 8)
        p_sum = total.data_ptr()
    y, ldy = _new_rows(x, rows, cols, dtype, 16)
    if dtype is _E4M3:
        scale = torch.empty(rows, dtype=_F32, device=x.device)
        p_scale = scale.data_ptr()
    check(_lib.load().eagle_rms_norm(x.data_ptr(), ldx, p_res, ldr, p_w, eps, rows, cols, p_sum, lds, _CODES[dtype], y.data_ptr(),
                                     ldy, p_scale, _stream(index)), "eagle_rms_norm")
    return y, scale, total


def linear_workspace(w, rows: int, stream=None):
    """Scratch for ``linear`` calls of up to `rows` rows on w's device, one call at a time: what makes large
    ones (over 1024 rows, some 20000 outputs) quicker whose ``out`` has rows that are not multiples of 16 bytes."""
    index = _device(w, "w")
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return linear_workspace(w, rows)
    nbytes = _lib.load().eagle_linear_epilogue_workspace_bytes(max(rows, 1))
    if nbytes == 0:
        raise ValueError(f"unusable number of rows ({rows})")
    ws = torch.empty(nbytes, dtype=_U8, device=w.device)
    ws[:_TICKETS].zero_()
    return ws


def linear(w, x, bias=None, act=None, residual=None, w_scale=None, x_scale=None, dtype=torch.bfloat16, out=None,
           workspace=None, stream=None):
    """y = act(w_scale x_scale (x w^T) + bias) + residual.  w [features][k] and x [rows][k] are bf16, or
    8-bit rows (float8_e4m3fn) with w_scale [features] and x_scale [rows] fp32; bias [features] bf16; act None,
    "silu", "gelu" or "swiglu" (w: gate rows, then as many up rows; y = silu(gate) up); residual [rows][out]
    bf16.  Returns y [rows][out] of dtype (bf16 or fp32), or fills out, which may be the residual.  workspace:
    one of ``linear_workspace``, or None; calls that may overlap need one each.  ``linear_status`` raises what a
    call could not do on the device."""
    code = _ACTS.get(act)
    if stream is None and code is not None:
        to = dtype if out is None else out.dtype
        if to is _BF16 or to is _F32:
            made = short.linear(w, x, bias, code, residual, w_scale, x_scale, to is _F32, out, workspace)
            if made is not NotImplemented:
                return made
    index = _device(w, "w")
    kind = w.dtype
    fp8 = kind is _E4M3
    if not fp8 and kind is not _BF16:
        raise TypeError(f"w must be torch.bfloat16 or torch.float8_e4m3fn, got {kind}")
    if code is None:
        raise ValueError(f"act must be one of None, 'silu', 'gelu', 'swiglu', got {act!r}")
    features, k, ldw = _rows(w, "w", kind, index)
    rows, xk, ldx = _rows(x, "x", kind, index)
    if xk != k:
        raise ValueError(f"x has {xk} columns, w {k}")
    width = features
    if code == 3:
        if features % 2:
            raise ValueError("swiglu needs as many up rows of w as gate rows")
        width = features // 2
    p_ws = p_xs = p_bias = p_res = p_work = None
    if fp8:
        if w_scale is None or x_scale is None:
            raise ValueError("8-bit operands have w_scale and x_scale")
        p_ws, p_xs = _vector(w_scale, "w_scale", _F32, index, features), _vector(x_scale, "x_scale", _F32, index, rows)
    elif w_scale is not None or x_scale is not None:
        raise ValueError("bf16 operands have no scales")
    if bias is not None:
        p_bias = _vector(bias, "bias", _BF16, index, features)
    ldr = nbytes = 0
    if residual is not None:
        r_rows, r_cols, ldr = _rows(residual, "residual", _BF16, index)
        if r_rows != rows or r_cols != width:
            raise ValueError(f"residual must be [{rows}][{width}]")
        p_res = residual.data_ptr()
    if out is not None:
        dtype = out.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"linear gives torch.bfloat16 or torch.float32, not {dtype}")
    if workspace is not None:
        if workspace.dtype is not _U8 or workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
        p_work, nbytes = workspace.data_ptr(), workspace.numel()
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return linear(w, x, bias, act, residual, w_scale, x_scale, dtype, out, workspace)
    if out is None:
        out, ldy = _new_rows(x, rows, width, dtype, 8)
    else:
        o_rows, o_cols, ldy = _rows(out, "out", dtype, index)
        if o_rows != rows or o_cols != width:
            raise ValueError(f"out must be [{rows}][{width}]")
    args = _lib.LinearArgs(rows, width, k, _CODES[kind], _CODES[dtype], code, w.data_ptr(), x.data_ptr(), ldw, ldx, p_ws, p_xs,
                           p_bias, p_res, ldr, out.data_ptr(), ldy)
    check(_lib.load().eagle_linear(ctypes.byref(args), p_work, nbytes, None, _stream(index)), "eagle_linear")
    return out


def linear_status(device=None, workspace=None, stream=None):
    """Waits for `stream` (default: the current one) of `device` (default: the current one, or the stream's), raises
    the first error that ``linear`` calls there have latched since the last call (a wait that ran out: the outputs
    of calls since then are undefined) and clears it.  workspace: one that such calls used; with an error it is
    made fit for use again."""
    if workspace is not None and workspace.dtype is not _U8:
        raise ValueError("workspace must be one of linear_workspace")
    if device is None:
        place = stream if stream is not None else workspace
        index = torch.cuda.current_device() if place is None else place.device.index
    else:
        device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"device must be a CUDA device, got {device}")
        index = torch.cuda.current_device() if device.index is None else device.index
    if workspace is not None and workspace.get_device() != index:
        raise ValueError(f"workspace is on {workspace.device}, not on cuda:{index}")
    with _elsewhere(index, stream) or _AS_IS:
        code = _lib.load().eagle_linear_status(_stream(index))
        if code != 0 and workspace is not None:
            workspace[:_TICKETS].zero_()
    check(code, "linear_status")


class DecoderLayerFP8:
    """The draft decoder layer in 8 bits over a 4-bit cache (eagle_decoder_layer_fp8_kv4).  Takes the bf16
    weights of ``DecoderLayer`` and keeps 8-bit rows of the projections': half the bytes.  They are ready when the
    constructor returns, for calls on any stream; the layer must live until its calls have ended."""

    def __init__(self, w_qkv, w_o, w_norm, w_gu, w_d, heads: int, kv_heads: int, rope_theta: float = 10000.0,
                 rms_eps: float = 1e-6):
        self._lib = _lib.load()
        for t, name in ((w_qkv, "w_qkv"), (w_o, "w_o"), (w_norm, "w_norm"), (w_gu, "w_gu"), (w_d, "w_d")):
            _need(t, name, _BF16, w_norm.device)
        h, inter = w_norm.shape[0], w_gu.shape[0] // 2
        D = w_qkv.shape[0] // (heads + 2 * kv_heads)
        if w_qkv.shape != (D * (heads + 2 * kv_heads), h) or w_o.shape != (h, heads * D) \
                or w_gu.shape != (2 * inter, h) or w_d.shape != (h, inter):
            raise ValueError("decoder layer weight shapes do not agree")
        if h % 16 or inter % 16:
            raise ValueError("hidden and inter must be multiples of 16")
        rows = [quantize_rows(t) for t in (w_qkv, w_o, w_gu, w_d)]
        with torch.cuda.device(w_norm.device):
            if not torch.cuda.is_current_stream_capturing():  # a graph's weights are ready when it has run
                torch.cuda.current_stream().synchronize()
        self._keep = (rows, w_norm)
        (qkv, s_qkv), (o, s_o), (gu, s_gu), (d, s_d) = ((c.data_ptr(), s.data_ptr()) for c, s in rows)
        self.w = _lib.DecoderLayerFP8Weights(h, heads, kv_heads, D, inter, rope_theta, rms_eps, qkv, o, w_norm.data_ptr(), gu, d,
                                             s_qkv, s_o, s_gu, s_d)
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.inter = h, heads, kv_heads, D, inter
        self.device = w_norm.device

    def workspace_bytes(self, cache, batch: int, nodes: int) -> int:
        """Bytes of scratch that a call with these sizes needs."""
        with cache._on(None):
            n = self._lib.eagle_decoder_layer_fp8_kv4_workspace_bytes(ctypes.byref(self.w), cache._ref, max(batch, 1), nodes)
        if n == 0:
            raise ValueError(f"unusable decoder layer sizes (batch={batch}, nodes={nodes}) or a cache of other heads")
        return n

    def kv4(self, x, cache, positions, mask=None, out=None, new_kv: bool = False, workspace=None, stream=None):
        """The layer over the cache, as ``DecoderLayer.kv4``: x [B][n][h] bf16, positions [B][n] int32, mask
        [B][n][ceil(n / 32)] int32 (None: node i sees nodes 0..i).  Returns out [B][n][h] bf16, and with new_kv
        the nodes' turned keys and values for ``cache.append``.  workspace: a uint8 tensor to use instead of a
        fresh one; calls that may overlap need one each."""
        _need(x, "x", _BF16)
        B, n, h = x.shape
        if h != self.hidden or B != cache.batch:
            raise ValueError("x does not match the weights or the cache")
        if cache.device != x.device or self.device != x.device:
            raise ValueError("the weights, the cache and x must be on one device")
        if _need(positions, "positions", torch.int32, x.device).shape != (B, n):
            raise ValueError("positions shape does not match")
        if mask is not None and _need(mask, "mask", torch.int32, x.device).shape != (B, n, (n + 31) // 32):
            raise ValueError("mask shape does not match")
        nbytes = self.workspace_bytes(cache, B, n)
        with cache._on(stream):
            if out is None:
                out = torch.empty_like(x)
            elif _need(out, "out", _BF16, x.device).shape != x.shape:
                raise ValueError("out shape does not match")
            kn = vn = p_kn = p_vn = None
            if new_kv:
                kn = torch.empty(B, n, self.kv_heads, self.head_dim, dtype=_BF16, device=x.device)
                vn = torch.empty_like(kn)
                p_kn, p_vn = kn.data_ptr(), vn.data_ptr()
            if workspace is None:
                workspace = torch.empty(nbytes, dtype=_U8, device=x.device)
            elif _need(workspace, "workspace", _U8, x.device).numel() < nbytes:
                raise ValueError(f"workspace must hold at least {nbytes} bytes")
            check(self._lib.eagle_decoder_layer_fp8_kv4(
                ctypes.byref(self.w), cache._ref, B, n, x.data_ptr(), positions.data_ptr(), None if mask is None else mask.data_ptr(),
                out.data_ptr(), p_kn, p_vn, workspace.data_ptr(), nbytes, cache._status.data_ptr(),
                cache._raw_stream(stream)), "eagle_decoder_layer_fp8_kv4")
        return (out, kn, vn) if new_kv else out
