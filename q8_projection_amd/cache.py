"""Python binding of include/q8_cache.h: the key/value cache and its attention.

As in the package's other wrappers, argument marshalling only.  Every tensor of
a call lives on one device, and the call runs on that device whichever is
current, on ``stream`` (a torch stream or a raw handle) or else on that device's
current stream.  Outputs and workspaces that are not passed are allocated here,
and cleared where that is needed, on the same stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

import q8_projection_amd as _q8

from .decode import _call, _need, _on_stream, _ptr

_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8


class _CacheC(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("pages", ctypes.c_int64), ("data", ctypes.c_void_p)]


class _BatchC(ctypes.Structure):
    _fields_ = [("sequences", ctypes.c_int64), ("table_ld", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("max_rows", ctypes.c_int64)]


def cache_page_bytes(bits: int, kv_heads: int, head_dim: int, page_tokens: int) -> int:
    """Bytes of a page of the cache (0: refused)."""
    c = _CacheC(bits, kv_heads, head_dim, page_tokens, 0, None)
    return int(_q8.lib().q8_cache_page_bytes(ctypes.addressof(c)))


class KVCache:
    """A pool of pages of one layer's keys and values, checked once.

    data: uint8 [pages][cache_page_bytes], used in place and kept alive by this object;
    or the number of pages, which are then allocated on ``device``.
    """

    def __init__(self, bits: int, kv_heads: int, head_dim: int, page_tokens: int, data, device=None):
        size = cache_page_bytes(bits, kv_heads, head_dim, page_tokens)
        if size == 0:
            raise ValueError(f"the library does not take this cache: {bits} bits, {kv_heads} heads of {head_dim}, "
                             f"pages of {page_tokens} tokens")
        if not isinstance(data, torch.Tensor):
            data = torch.empty((int(data), size), dtype=_U8, device=device or torch.device("cuda"))
        if data.dim() != 2 or not data.is_cuda:
            raise ValueError("data must be a device tensor [pages][cache_page_bytes]")
        self.device = data.device
        _need(data, "data", _U8, (data.shape[0], size), self.device)
        self.bits, self.kv_heads, self.head_dim, self.page_tokens = bits, kv_heads, head_dim, page_tokens
        self.pages, self.data = data.shape[0], data
        if not 1 <= self.pages < 1 << 31:
            raise ValueError(f"{self.pages} pages: 1 to 2^31 - 1 are taken")
        self._c = _CacheC(bits, kv_heads, head_dim, page_tokens, self.pages, data.data_ptr())
        self._ref = ctypes.addressof(self._c)


class CacheBatch:
    """The sequences of calls on a cache, checked once.

    table: int32 [sequences][entries], the pages of each sequence; lens: int32
    [sequences], its tokens, the rows of the call included; starts: int32 [sequences + 1],
    the rows of each sequence, or None: a row a sequence.  rows: rows of the calls' arrays
    (with ``starts``; else as many as sequences); max_rows: rows of one sequence at most
    (None: ``rows``).  The tensors are used in place: a loop that changes their contents
    keeps the object.  Rows behind the last sequence and those of a sequence past
    ``max_rows`` belong to none: calls neither take them nor write them, and do not say so.
    """

    def __init__(self, cache: KVCache, table: torch.Tensor, lens: torch.Tensor, starts=None, rows=None, max_rows=None):
        if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[1] < 1:
            raise ValueError("table must be an int32 tensor [sequences][entries]")
        n = table.shape[0]
        _need(table, "table", _I32, table.shape, cache.device)
        _need(lens, "lens", _I32, (n,), cache.device)
        if starts is not None:
            _need(starts, "starts", _I32, (n + 1,), cache.device)
            if rows is None:
                raise ValueError("rows is required with starts")
        elif rows is not None and rows != n:
            raise ValueError(f"rows must be the number of sequences ({n}) without starts, not {rows}")
        self.rows = n if starts is None else int(rows)
        self.max_rows = max(1, self.rows if max_rows is None else int(max_rows)) if starts is not None else 1
        self.device = cache.device
        self._tensors = (table, lens, starts)
        self._c = _BatchC(n, table.shape[1], table.data_ptr(), lens.data_ptr(), _ptr(starts), self.rows, self.max_rows)
        self._ref = ctypes.addressof(self._c)
        self._bytes = {}

    def _workspace_bytes(self, cache, heads: int) -> int:
        key = (cache.kv_heads, cache.head_dim, cache.page_tokens, cache.bits, heads)
        if key not in self._bytes:
            with torch.cuda.device(self.device):
                self._bytes[key] = int(_q8.lib().q8_attention_workspace_bytes(cache._ref, self._ref, heads))
        return self._bytes[key]


def _rows_of(t, name, cache, batch, heads=None):
    """(heads, row stride) of f32 rows [rows][heads][head_dim], a view whose rows may lie apart."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.dtype != _F32 or t.device != cache.device:
        raise ValueError(f"{name} must be a f32 tensor [rows][heads][head_dim] on {cache.device}")
    rows, h, d = t.shape
    if rows != batch.rows or d != cache.head_dim or (heads is not None and h != heads):
        raise ValueError(f"{name} must have shape {(batch.rows, heads or 'heads', cache.head_dim)}, not {tuple(t.shape)}")
    ld, sh, sd = t.stride()
    if rows and h and (sd != 1 or (h > 1 and sh != d)):
        raise ValueError(f"{name} must be contiguous within a row")
    return h, ld if rows > 1 else h * d


def _same(cache, batch):
    if batch.device != cache.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")


def cache_append(cache: KVCache, batch: CacheBatch, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Write the rows' keys and values, f32 [rows][kv_heads][head_dim] (views of a wider
    buffer's columns too), into the cache; rows of no sequence (``CacheBatch``) are not written.

    Sequences of the batch may write to the same pages, but no two rows to the same token's place.
    """
    if stream is not None:
        return _on_stream(stream, cache.device, cache_append, cache, batch, k, v)
    _same(cache, batch)
    _, k_ld = _rows_of(k, "k", cache, batch, cache.kv_heads)
    _, v_ld = _rows_of(v, "v", cache, batch, cache.kv_heads)
    _call("q8_cache_append", cache.device, batch.rows, cache._ref, batch._ref, k.data_ptr(), k_ld, v.data_ptr(), v_ld)


def _out(t, name, shape, device):
    if t is None:
        return torch.empty(shape, dtype=_F32, device=device)
    _need(t, name, _F32, shape, device)
    return t


def cache_read(cache: KVCache, batch: CacheBatch, k=None, v=None, stream=None):
    """(k, v) f32 [rows][kv_heads][head_dim]: the values that the cache stands for at the rows' tokens.

    Rows of no sequence (``CacheBatch``) are left as they were: in outputs that are allocated here, arbitrary.
    """
    if stream is not None:
        return _on_stream(stream, cache.device, cache_read, cache, batch, k, v)
    _same(cache, batch)
    shape = (batch.rows, cache.kv_heads, cache.head_dim)
    k, v = _out(k, "k", shape, cache.device), _out(v, "v", shape, cache.device)
    _call("q8_cache_read", cache.device, batch.rows, cache._ref, batch._ref, k.data_ptr(), v.data_ptr())
    return k, v


def attention_workspace_bytes(cache: KVCache, batch: CacheBatch, heads: int) -> int:
    """Bytes of the attention's workspace (0: refused)."""
    _same(cache, batch)
    return batch._workspace_bytes(cache, int(heads))


def attention_workspace(cache: KVCache, batch: CacheBatch, heads: int) -> torch.Tensor:
    """A zero-filled workspace for the attention of `heads` query heads over this batch."""
    return torch.zeros(attention_workspace_bytes(cache, batch, heads), dtype=_U8, device=cache.device)


def attention(cache: KVCache, batch: CacheBatch, q: torch.Tensor, scale=None, window: int = 0, out=None, lse=None,
              workspace=None, stream=None):
    """(out f32 [rows][heads][head_dim], lse f32 [rows][heads]) of the queries q, f32
    [rows][heads][head_dim] (a view of a wider buffer's columns too), over the cache.

    scale: 1 / sqrt(head_dim) if None; window: tokens that a row sees at most, itself
    among them (0: all before it).  The workspace (uint8, zero-filled, at least
    attention_workspace_bytes) may be kept from call to call; without one, one is allocated and
    all of it cleared in each call, up to 52 MB (2 to 14 us more).  Rows of no sequence (``CacheBatch``) are
    left as they were: in outputs that are allocated here, arbitrary.
    """
    if stream is not None:
        return _on_stream(stream, cache.device, attention, cache, batch, q, scale, window, out, lse, workspace)
    _same(cache, batch)
    heads, q_ld = _rows_of(q, "q", cache, batch)
    dev = cache.device
    out = _out(out, "out", (batch.rows, heads, cache.head_dim), dev)
    lse = _out(lse, "lse", (batch.rows, heads), dev)
    if workspace is None:
        workspace = attention_workspace(cache, batch, heads)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != _U8 or workspace.device != dev or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the cache's device")
    if scale is None:
        scale = 1.0 / math.sqrt(cache.head_dim)
    _call("q8_attention", dev, batch.rows, cache._ref, batch._ref, q.data_ptr(), q_ld, heads, scale, window,
          out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse
