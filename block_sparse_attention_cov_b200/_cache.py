"""Key/value cache in 8 bits with a scale per 64-token block and head (solattn_cache_append, solattn_cache_attention)."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from . import _check, _current, _dtype, _ptr, _same_device, _shape, _stream_on, _tensor_strides

__all__ = ["Cache", "cache_append", "cache_workspace", "cache_attention"]


class Cache:
    """Pages of a cache: k, v float8_e4m3fn [pages, heads, 64, d] and float32 scales [pages, heads], the tensors that
    the calls read and write (any step between pages, as in a slice of a cache of several layers). A value is
    k[p, h, t] * k_scale[p, h]. Cache.empty() makes them; which page holds what is the caller's table."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        for x in (k, v):
            if not x.is_cuda or x.dtype != torch.float8_e4m3fn or x.dim() != 4 or x.shape[2] != _lib.BLOCK:
                raise ValueError("k, v must be CUDA float8_e4m3fn [pages, heads, 64, d] tensors")
        for x in (k_scale, v_scale):
            if x.dtype != torch.float32 or tuple(x.shape) != tuple(k.shape[:2]):
                raise ValueError("k_scale, v_scale must be float32 [pages, heads]")
        _same_device(k, v, k_scale, v_scale)
        pages, heads, _, d = k.shape
        inner = (_lib.BLOCK * d, d, 1)
        if v.shape != k.shape or v.stride() != k.stride() or k_scale.stride() != v_scale.stride():
            raise ValueError("keys and values must share their shapes and strides")
        if pages == 0 or heads == 0:
            raise ValueError("a cache needs a page and a head")
        if (heads > 1 and k.stride(0 + 1) != inner[0]) or k.stride()[2:] != inner[1:]:
            raise ValueError("a page must be contiguous [heads, 64, d]")
        if heads > 1 and k_scale.stride(1) != 1:
            raise ValueError("a page's scales must be adjacent")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.d = int(pages), int(heads), int(d)
        many = pages > 1
        self.struct = _lib.CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads,
                                       d, k.stride(0) if many else 0, k_scale.stride(0) if many else 0)

    @classmethod
    def empty(cls, pages: int, heads: int, d: int, device=None) -> "Cache":
        """A cache of unwritten pages (no sequence may read a token before it was appended)."""
        device = torch.device("cuda" if device is None else device)
        k, v = (torch.empty((pages, heads, _lib.BLOCK, d), dtype=torch.float8_e4m3fn, device=device) for _ in range(2))
        ks, vs = (torch.empty((pages, heads), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def _check_table(cache, table, lengths, counts, B):
    _same_device(cache.k, table, lengths, counts)
    if table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != B or table.shape[1] < 1:
        raise ValueError("table must be int32 [B, columns]")
    if table.shape[1] > 1 and table.stride(1) != 1 or (B > 1 and table.stride(0) < table.shape[1]):
        raise ValueError("a row of the table must be contiguous, rows apart")
    for x, name in ((lengths, "lengths"), (counts, "counts")):
        if x is not None and (x.dtype != torch.int32 or tuple(x.shape) != (B,) or (B > 1 and x.stride(0) != 1)):
            raise ValueError(f"{name} must be contiguous int32 [B]")
    return int(table.shape[1]), table.stride(0) if B > 1 else 0


def _check_status(ws, need):
    if ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous() or ws.numel() < need:
        raise ValueError(f"ws must be a contiguous CUDA uint8 tensor of at least {need} bytes")


def cache_append(cache: Cache, k, v, table, lengths, counts=None, ws=None) -> None:
    """Writes the keys and values k, v [B, heads, N, d] (bf16, fp16 or fp32; one set of strides, d contiguous) of
    counts[b] (None: N) new tokens behind the lengths[b] tokens that sequence b has in the cache; lengths itself is the
    caller's and does not change. table int32 [B, columns]: the page of each 64-token block; a page that is written
    belongs to one sequence. ws: a workspace (workspace() or cache_workspace()) whose status() then reports
    a page or length out of range."""
    B, H, N, d = _shape(k)
    for x in (k, v):
        if not (x.is_cuda and x.dim() == 4 and x.stride(-1) == 1):
            raise ValueError("k, v must be CUDA [B, heads, N, d] tensors with contiguous d")
    if v.shape != k.shape or v.dtype != k.dtype or v.stride() != k.stride():
        raise ValueError("k and v must share their shape, type and strides")
    if (H, d) != (cache.heads, cache.d):
        raise ValueError("k, v do not match the cache's heads and d")
    dtype = _dtype(k, fp32=True)
    _same_device(k, v, cache.k, ws)
    columns, table_stride = _check_table(cache, table, lengths, counts, B)
    if ws is not None:
        _check_status(ws, _lib.WORKSPACE_BYTES)
    with _current(k):
        _check(_lib.lib().solattn_cache_append(_ptr(k), _ptr(v), dtype, B, N, _tensor_strides(k), cache.struct,
                                               _ptr(table), columns, table_stride, _ptr(lengths), _ptr(counts), _ptr(ws),
                                               0 if ws is None else ws.numel(), _stream_on(k)), "solattn_cache_append")


def _workspace_bytes(B, H, N, d, heads, columns) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.lib().solattn_cache_workspace_bytes(B, H, N, d, heads, columns, ctypes.byref(n)),
           "solattn_cache_workspace_bytes")
    return int(n.value)


def cache_workspace(q, cache: Cache, table) -> torch.Tensor:
    """A workspace for cache_attention() of these sizes, its status cleared."""
    B, H, N, d = _shape(q)
    ws = torch.empty(_workspace_bytes(B, H, N, d, cache.heads, int(table.shape[1])), dtype=torch.uint8, device=q.device)
    ws[:_lib.WORKSPACE_BYTES].zero_()
    return ws


def cache_attention(q, cache: Cache, table, lengths, counts=None, causal: bool = True, scale: float | None = None,
                    out=None, lse=None, ws=None, want_lse: bool = True):
    """Softmax attention of q [B, H, N, d] (bf16 or fp16) over the cache. Returns (out, lse).

    H is a multiple of cache.heads; lengths int32 [B] counts each sequence's tokens in the cache, its queries' own
    among them; counts int32 [B] (None: N) of the N query rows are there and stand for the sequence's last tokens. causal: a
    query sees the keys up to its own place, else all of the sequence's. scale: 1/sqrt(d) when None. A row that sees no
    key gives 0 and -inf; rows behind counts[b] keep what out and lse held (torch.empty when allocated here). ws: from
    cache_workspace(), kept by the caller for status(ws) and for graphs; allocated here when None."""
    if not (q.is_cuda and q.dim() == 4 and q.stride(-1) == 1):
        raise ValueError("q must be a CUDA [B, H, N, d] tensor with contiguous d")
    dtype = _dtype(q, fp32=False)
    B, H, N, d = _shape(q)
    if d != cache.d or H % cache.heads:
        raise ValueError("q does not match the cache's heads and d")
    columns, table_stride = _check_table(cache, table, lengths, counts, B)
    if scale is not None and not (math.isfinite(scale) and scale > 0):
        raise ValueError("scale must be positive and finite")
    out = torch.empty_like(q) if out is None else out
    if out.shape != q.shape or out.dtype != q.dtype or out.stride(-1) != 1:
        raise ValueError("out must have q's shape and type and a contiguous d")
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    _same_device(q, cache.k, out, lse, ws)
    with _current(q):
        if ws is None:
            ws = cache_workspace(q, cache, table)
        else:
            _check_status(ws, _lib.WORKSPACE_BYTES)
        _check(_lib.lib().solattn_cache_attention(_ptr(q), dtype, B, H, N, d, _tensor_strides(q), cache.struct, _ptr(table),
                                                  columns, table_stride, _ptr(lengths), _ptr(counts), int(bool(causal)),
                                                  0.0 if scale is None else float(scale), _ptr(out), _tensor_strides(out),
                                                  _ptr(lse), _ptr(ws), ws.numel(), _stream_on(q)),
               "solattn_cache_attention")
    return out, lse
