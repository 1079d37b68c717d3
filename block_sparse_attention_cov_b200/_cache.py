"""Key/value cache in 8 bits with a scale per 64-token block and head (solattn_cache_append, solattn_cache_attention)."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from . import _CODES16, _at, _call, _check, _device_index, _dtype, _tensor_strides

__all__ = ["Cache", "cache_append", "cache_workspace", "cache_attention"]


class Cache:
    """Pages of a cache: k, v float8_e4m3fn [pages, heads, 64, d] and float32 scales [pages, heads] (2^-32 .. 2^32), the
    tensors that the calls read and write (any step between pages, as in a slice of a cache of several layers). A value is
    k[p, h, t] * k_scale[p, h]. Cache.empty() makes them; which page holds what is the caller's table. The tensors are
    written in place, never replaced: the calls use the addresses that they had when the Cache was made."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        for x in (k, v):
            if not x.is_cuda or x.dtype != torch.float8_e4m3fn or x.dim() != 4 or x.shape[2] != _lib.BLOCK:
                raise ValueError("k, v must be CUDA float8_e4m3fn [pages, heads, 64, d] tensors")
        for x in (k_scale, v_scale):
            if x.dtype != torch.float32 or tuple(x.shape) != tuple(k.shape[:2]):
                raise ValueError("k_scale, v_scale must be float32 [pages, heads]")
        self._dev = _device_index(k, v, k_scale, v_scale)
        pages, heads, _, d = k.shape
        inner = (_lib.BLOCK * d, d, 1)
        if v.shape != k.shape or v.stride() != k.stride() or k_scale.stride() != v_scale.stride():
            raise ValueError("keys and values must share their shapes and strides")
        if pages == 0 or heads == 0:
            raise ValueError("a cache needs a page and a head")
        if (heads > 1 and k.stride(1) != inner[0]) or k.stride()[2:] != inner[1:]:
            raise ValueError("a page must be contiguous [heads, 64, d]")
        if heads > 1 and k_scale.stride(1) != 1:
            raise ValueError("a page's scales must be adjacent")
        if pages > 1 and (k.stride(0) < heads * inner[0] or k_scale.stride(0) < heads):
            raise ValueError("pages, and their scales, must be apart (not expand()ed from one)")
        self._tensors = (k, v, k_scale, v_scale)
        self.pages, self.heads, self.d = int(pages), int(heads), int(d)
        many = pages > 1
        self.struct = _lib.CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads,
                                       d, k.stride(0) if many else 0, k_scale.stride(0) if many else 0)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    def __reduce__(self):  # copies are made of the tensors, with their addresses
        return Cache, self._tensors

    @classmethod
    def empty(cls, pages: int, heads: int, d: int, device=None) -> "Cache":
        """A cache of unwritten pages (no sequence may read a token before it was appended)."""
        device = torch.device("cuda" if device is None else device)
        k, v = (torch.empty((pages, heads, _lib.BLOCK, d), dtype=torch.float8_e4m3fn, device=device) for _ in range(2))
        ks, vs = (torch.empty((pages, heads), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def _check_table(table, lengths, counts, B: int):
    """(columns, step between rows) of the table."""
    if table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table must be int32 [B, columns]")
    columns, (step, inner) = table.shape[1], table.stride()
    if columns < 1 or (columns > 1 and inner != 1) or (B > 1 and step < columns):
        raise ValueError("a row of the table must be contiguous, rows apart")
    for x in (lengths, counts):
        if x is not None and (x.dtype != torch.int32 or x.dim() != 1 or x.shape[0] != B or (B > 1 and x.stride(0) != 1)):
            raise ValueError("lengths and counts must be contiguous int32 [B]")
    return columns, step if B > 1 else 0


def _check_workspace(ws):
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor")
    return ws.numel()


def cache_append(cache: Cache, k, v, table, lengths, counts=None, ws=None) -> None:
    """Writes the keys and values k, v [B, heads, N, d] (bf16, fp16 or fp32; one set of strides, d contiguous) of
    counts[b] (None: N) new tokens behind the lengths[b] tokens that sequence b has in the cache; lengths itself is the
    caller's and does not change. table int32 [B, columns]: the page of each 64-token block; a page that is written
    belongs to one sequence. ws: a workspace, cleared once (cache_workspace(), or workspace().zero_()), whose status()
    then reports a page, length or count out of range."""
    if k.dim() != 4 or k.stride(3) != 1:
        raise ValueError("k, v must be [B, heads, N, d] tensors with contiguous d")
    if v.shape != k.shape or v.dtype != k.dtype or v.stride() != k.stride():
        raise ValueError("k and v must share their shape, type and strides")
    B, H, N, d = k.shape
    if H != cache.heads or d != cache.d:
        raise ValueError("k, v do not match the cache's heads and d")
    dtype = _dtype(k)
    columns, step = _check_table(table, lengths, counts, B)
    dev = _device_index(cache.k, k, v, table, lengths, counts, ws)
    _call("solattn_cache_append", _lib.lib().solattn_cache_append, dev, k.data_ptr(), v.data_ptr(), dtype, B, N,
          _tensor_strides(k), cache.struct, table.data_ptr(), columns, step, lengths.data_ptr(), _at(counts), _at(ws),
          0 if ws is None else _check_workspace(ws))


@functools.lru_cache(maxsize=512)
def _workspace_bytes(B: int, H: int, N: int, d: int, heads: int, columns: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.lib().solattn_cache_workspace_bytes(B, H, N, d, heads, columns, ctypes.byref(n)),
           "solattn_cache_workspace_bytes")
    return int(n.value)


def cache_workspace(q, cache: Cache, table) -> torch.Tensor:
    """A workspace for cache_attention() of these sizes, its status cleared. Its bytes follow how the call is split and may
    fall where a size grows: for calls of several sizes keep the largest of their workspaces."""
    B, H, N, d = q.shape
    ws = torch.empty(_workspace_bytes(B, H, N, d, cache.heads, table.shape[1]), dtype=torch.uint8, device=q.device)
    ws[:_lib.WORKSPACE_BYTES].zero_()
    return ws


def cache_attention(q, cache: Cache, table, lengths, counts=None, causal: bool = True, scale: float | None = None,
                    out=None, lse=None, ws=None, want_lse: bool = True):
    """Softmax attention of q [B, H, N, d] (bf16 or fp16) over the cache. Returns (out, lse).

    H is a multiple of cache.heads; lengths int32 [B] counts each sequence's tokens in the cache, its queries' own
    among them; counts int32 [B] (None: N) of the N query rows are there and stand for the sequence's last tokens.
    causal: a query sees the keys up to its own place, else all of the sequence's. scale: 1/sqrt(d) when None. A row that
    sees no key gives 0 and -inf; rows behind counts[b] keep what out and lse held (torch.empty when allocated here).
    ws: from cache_workspace(), kept by the caller for status(ws) and for graphs; allocated here when None, and then
    nobody learns of a page, length or count out of range (tokens of such a page are left out, lengths clamped)."""
    if q.dim() != 4 or q.stride(3) != 1:
        raise ValueError("q must be a [B, H, N, d] tensor with contiguous d")
    dtype = _dtype(q, _CODES16)
    if q.get_device() < 0:
        raise ValueError("expected CUDA tensors")
    B, H, N, d = q.shape
    if d != cache.d or H % cache.heads:
        raise ValueError("q does not match the cache's heads and d")
    columns, step = _check_table(table, lengths, counts, B)
    if scale is None:
        scale = 0.0
    elif not 0.0 < ctypes.c_float(scale).value < 2.0 ** 127:
        raise ValueError("scale must be positive and below 2^127 in fp32")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.stride(3) != 1:
        raise ValueError("out must have q's shape and type and a contiguous d")
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if want_lse else None
    elif lse.dtype != torch.float32 or lse.shape != q.shape[:3] or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    if ws is None:
        ws = cache_workspace(q, cache, table)
    dev = _device_index(q, cache.k, table, lengths, counts, out, lse, ws)
    _call("solattn_cache_attention", _lib.lib().solattn_cache_attention, dev, q.data_ptr(), dtype, B, H, N, d,
          _tensor_strides(q), cache.struct, table.data_ptr(), columns, step, lengths.data_ptr(), _at(counts),
          1 if causal else 0, scale, out.data_ptr(), _tensor_strides(out), _at(lse), ws.data_ptr(), _check_workspace(ws))
    return out, lse
