"""A key/value cache in 4 bits: argument marshalling over the eagle_kv4_* entry points of the C ABI.

One round of drafting with it: the decoder layer attends over the cache (``DecoderLayer.kv4``, or
``KV4Cache.attention`` alone) and hands out the keys and values of the tree's nodes; the verify names
the accepted nodes; ``KV4Cache.append`` quantises those nodes' rows into the cache.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import EAGLE_BF16, EAGLE_F32, check
from .engine import _need

_BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8
_DTYPES = {torch.bfloat16: EAGLE_BF16, torch.float32: EAGLE_F32}
_AS_IS = contextlib.nullcontext()


def _here(t, name, device, dtype=None):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _ints(t, name, device, shape):
    """The address of a contiguous int32 tensor of this shape, or None."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype is not _I32 or t.get_device() != device.index:
        _here(t, name, device, _I32)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _row_step(t, name):
    """Elements between the rows of a [B][n][heads][D] tensor whose rows are packed (a contiguous
    tensor, or a slice of wider rows such as a projection's output)."""
    B, n, h, D = t.shape
    row = h * D
    if t.is_contiguous():
        return row  # whatever the strides of sizes of 1
    if t.stride(3) != 1 or (h > 1 and t.stride(2) != D):
        raise ValueError(f"{name}: a row's heads must be packed")
    step = t.stride(1) if n > 1 else (t.stride(0) if B > 1 else row)
    if n > 1 and B > 1 and t.stride(0) != n * step:
        raise ValueError(f"{name}: rows of all requests must be evenly spaced")
    if step < row or step % 8:
        raise ValueError(f"{name}: rows must be a multiple of 8 elements apart and not overlap")
    return step


class KV4Cache:
    """A paged 4-bit cache of `batch` requests (see eagle_kv4_cache in include/eagle_tree.h).

    table [batch][max_pages] int32 and lengths [batch] int32 are the cache's own tensors: a scheduler
    writes page numbers into `table` (it starts as pages 0, 1, 2, ... dealt out request by request
    where the pool is large enough, else as -1) and may set `lengths` (they start as 0).  page_size is
    a power of two of at least 16; head_dim 32, 64, 96 or 128."""

    def __init__(self, batch: int, kv_heads: int, head_dim: int, num_pages: int, max_pages: int,
                 page_size: int = 64, device=None, pages=None):
        self._lib = _lib.load()
        self.device = torch.device("cuda" if device is None else device)
        if self.device.type != "cuda":
            raise ValueError("a KV4Cache lives on a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self.batch, self.kv_heads, self.head_dim = batch, kv_heads, head_dim
        self._tail = (kv_heads, head_dim)
        self.page_size, self.num_pages, self.max_pages = page_size, num_pages, max_pages
        self._c = _lib.KV4CacheStruct(kv_heads, head_dim, page_size, num_pages, max_pages, None, None, None)
        self._ref = ctypes.byref(self._c)
        nbytes = self._lib.eagle_kv4_pages_bytes(self._ref)
        if nbytes == 0 or batch < 1:
            raise ValueError("unusable 4-bit cache sizes")
        if pages is None:
            pages = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        elif _need(_here(pages, "pages", self.device, _U8), "pages").numel() < nbytes:
            raise ValueError(f"pages must hold at least {nbytes} bytes")
        self._pages = pages
        if num_pages >= batch * max_pages:
            self._table = torch.arange(batch * max_pages, dtype=torch.int32, device=self.device).view(batch, max_pages)
        else:
            self._table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=self.device)
        self._lengths = torch.zeros(batch, dtype=torch.int32, device=self.device)
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._c.pages, self._c.table, self._c.lengths = pages.data_ptr(), self._table.data_ptr(), self._lengths.data_ptr()
        self._status_ptr = self._status.data_ptr()
        self._plans = {}

    pages = property(lambda self: self._pages, doc="The page pool, uint8.")
    table = property(lambda self: self._table, doc="Pages of each request, [batch][max_pages] int32.")
    lengths = property(lambda self: self._lengths, doc="Positions held, [batch] int32.")
    capacity = property(lambda self: self.max_pages * self.page_size, doc="Positions a request can hold.")

    def _on(self, stream):
        """Makes the cache's device current, and `stream` where one is given, so that what is
        allocated belongs to the stream that uses it."""
        if stream is not None:
            if stream.device != self.device:
                raise ValueError(f"stream is on {stream.device}, the cache on {self.device}")
            return torch.cuda.stream(stream)
        if torch.cuda.current_device() != self._index:
            return torch.cuda.device(self.device)
        return _AS_IS

    def _raw_stream(self, stream):
        return torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream

    def _kv(self, k, v):
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype is not _BF16 or t.get_device() != self._index:
                _here(t, name, self.device, _BF16)
            if t.dim() != 4 or t.shape[0] != self.batch or t.shape[2:] != self._tail:
                raise ValueError(f"{name} must be [{self.batch}][rows][{self.kv_heads}][{self.head_dim}]")
        if k.shape != v.shape:
            raise ValueError("k and v must have the same shape")
        if k.shape[1] == 0:
            return self.kv_heads * self.head_dim
        ld = _row_step(k, "k")
        if _row_step(v, "v") != ld:
            raise ValueError("k and v must have the same row spacing")
        return ld

    def append(self, k, v, select=None, count=None, start=None, stream=None):
        """Quantises rows of k and v ([batch][rows][kv_heads][head_dim] bf16) into the cache, behind
        each request's length or from start [batch] int32 on, and sets the lengths to the end of
        what was written.  select [batch][slots] int32 names the row of each slot (negative: the slot
        is not written), e.g. a verify's accept_nodes; count [batch] int32 is each request's number of
        slots."""
        ld = self._kv(k, v)
        slots = rows = k.shape[1]
        if select is not None:
            if select.dim() != 2:
                raise ValueError("select must be [batch][slots]")
            slots = select.shape[1]
        # addresses beside the tensors, which must live until the call is enqueued
        p_select = _ints(select, "select", self.device, (self.batch, slots))
        p_count = _ints(count, "count", self.device, (self.batch,))
        p_start = _ints(start, "start", self.device, (self.batch,))
        with self._on(stream):
            check(self._lib.eagle_kv4_append(self._ref, self.batch, rows, slots, k.data_ptr(), v.data_ptr(), ld, p_select,
                                             p_count, p_start, self._status_ptr, self._raw_stream(stream)), "eagle_kv4_append")

    def read(self, start=None, rows=None, dtype=torch.bfloat16, out=None, stream=None):
        """The values that positions start[b] (default 0) .. + rows - 1 stand for: (k, v), each
        [batch][rows][kv_heads][head_dim] of `dtype` (bf16 or fp32).  out = (k, v) receives them (its
        shape gives rows); rows behind a request's length are left as they are (0 in fresh
        tensors).  rows defaults to the capacity."""
        p_start = _ints(start, "start", self.device, (self.batch,))
        with self._on(stream):
            if out is None:
                shape = (self.batch, self.capacity if rows is None else rows, *self._tail)
                out = (torch.zeros(shape, dtype=dtype, device=self.device), torch.zeros(shape, dtype=dtype, device=self.device))
            k, v = out
            for t, name in ((k, "out[0]"), (v, "out[1]")):
                if not _here(t, name, self.device).is_contiguous() or t.dtype not in _DTYPES:
                    raise ValueError(f"{name} must be a contiguous bf16 or fp32 tensor")
                if t.dim() != 4 or t.shape[0] != self.batch or t.shape[2:] != self._tail:
                    raise ValueError(f"{name} must be [{self.batch}][rows][{self.kv_heads}][{self.head_dim}]")
            if k.shape != v.shape or k.dtype != v.dtype or (rows is not None and k.shape[1] != rows):
                raise ValueError("the outputs must agree in shape and dtype")
            check(self._lib.eagle_kv4_read(self._ref, self.batch, k.shape[1], p_start, k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype],
                                           self._status_ptr, self._raw_stream(stream)), "eagle_kv4_read")
        return k, v

    def attention_workspace_bytes(self, nodes: int, heads: int) -> int:
        """Bytes of scratch that an attention call with these sizes needs."""
        with self._on(None):
            n = self._lib.eagle_kv4_attention_workspace_bytes(self._ref, nodes, heads)
        if n == 0:
            raise ValueError(f"unusable attention sizes (nodes={nodes}, heads={heads})")
        return n

    def _plan(self, q):
        """What an attention call with queries of this shape needs: checked and computed once."""
        if q.dim() != 4 or q.shape[0] != self.batch or q.shape[3] != self.head_dim or q.shape[1] < 1:
            raise ValueError(f"q must be [{self.batch}][n][heads][{self.head_dim}]")
        n, heads = q.shape[1], q.shape[2]
        plan = (n, heads, self.attention_workspace_bytes(n, heads), (self.batch, n, *self._tail),
                (self.batch, n, (n + 31) // 32), heads * self.head_dim, self.kv_heads * self.head_dim)
        self._plans[q.shape] = plan
        return plan

    def attention(self, q, k=None, v=None, mask=None, out=None, workspace=None, stream=None):
        """Attention of the nodes' queries q [batch][n][heads][head_dim] bf16 over each request's
        cached positions and the nodes' new keys and values k, v [batch][n][kv_heads][head_dim]:
        those that mask [batch][n][ceil(n / 32)] int32 marks, or without a mask the node's own and
        the earlier ones.  Returns out [batch][n][heads][head_dim] bf16.  workspace: a uint8 tensor to
        use instead of a fresh one; calls that may overlap need one each."""
        shape = q.shape
        n, heads, nbytes, kv_shape, mask_shape, ldq, ldkv = self._plans.get(shape) or self._plan(q)
        if q.dtype is not _BF16 or q.get_device() != self._index:
            _here(q, "q", self.device, _BF16)
        if not q.is_contiguous():
            ldq = _row_step(q, "q")
        p_k = p_v = p_mask = None
        if k is not None and v is not None:
            if k.shape != kv_shape or v.shape != kv_shape:
                raise ValueError(f"k and v must be {list(kv_shape)}")
            if not (k.dtype is v.dtype is _BF16 and k.get_device() == v.get_device() == self._index and k.is_contiguous()
                    and v.is_contiguous()):
                ldkv = self._kv(k, v)
            p_k, p_v = k.data_ptr(), v.data_ptr()
        elif k is not v:
            raise ValueError("k and v go together")
        elif mask is not None:
            raise ValueError("a mask needs k and v")
        if mask is not None:
            p_mask = _ints(mask, "mask", self.device, mask_shape)
        with self._on(stream):
            if out is None:
                out = q.new_empty(shape)
            elif not _here(out, "out", self.device, _BF16).is_contiguous() or out.shape != shape:
                raise ValueError("out must be contiguous and have the shape of q")
            if workspace is None:
                workspace = self._pages.new_empty(nbytes)
            elif _need(_here(workspace, "workspace", self.device, _U8), "workspace").numel() < nbytes:
                raise ValueError(f"workspace must hold at least {nbytes} bytes")
            check(self._lib.eagle_kv4_attention(self._ref, self.batch, n, heads, q.data_ptr(), ldq, p_k, p_v, ldkv, p_mask,
                                                out.data_ptr(), workspace.data_ptr(), nbytes, self._status_ptr,
                                                self._raw_stream(stream)), "eagle_kv4_attention")
        return out

    def status(self, stream=None):
        """Waits for `stream` (default: the current one), raises the first device error latched since
        the last call (an index out of range, a wait that ran out) and clears it."""
        with self._on(stream):
            bits = int(self._status.item())
            if bits:
                self._status.zero_()
        check(5 if bits & 1 else (6 if bits else 0), "KV4Cache.status")
