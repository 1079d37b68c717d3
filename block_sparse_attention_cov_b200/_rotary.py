"""Rotary positions on queries and keys (solattn_rotary, solattn_rotary_pool)."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from . import (PooledStats, _check, _check_inputs, _current, _dtype, _pooled_stats, _ptr, _same_device, _shape,
               _stream_on, _strides, _tensor_strides)

__all__ = ["Rotary", "rotary", "rotary_pool"]

LAYOUTS = {"interleaved": _lib.ROTARY_INTERLEAVED, "half": _lib.ROTARY_HALF}
SCALINGS = {"linear": _lib.SCALING_LINEAR, "ntk": _lib.SCALING_NTK, "yarn": _lib.SCALING_YARN}


class Rotary:
    """The frequencies of a rotary embedding, on the device, made once and used by every call.

    rot: rotated leading elements of a head (even). layout: "half" (element p pairs with p + rot/2) or "interleaved"
    (2p with 2p + 1). sections: rotated pairs of each position axis (for video, t, h and w), each with frequencies
    theta^(-i / n) of its own; None: one axis. scaling: None, ("linear", factor), ("ntk", factor) or
    ("yarn", factor, original_length[, fast, slow]). frequencies: rot / 2 values in radians per position that replace
    all of theta and scaling (pairs keep their axes)."""

    def __init__(self, rot: int, layout: str = "half", theta: float = 10000.0, sections=None, scaling=None,
                 frequencies=None, gain: float | None = None, device=None):
        if layout not in LAYOUTS:
            raise ValueError(f"unknown layout {layout!r}")
        rot = int(rot)
        if rot <= 0 or rot % 2:
            raise ValueError("rot must be positive and even")
        pairs = [rot // 2] if sections is None else [int(n) for n in sections]
        axes = len(pairs)
        if not 1 <= axes <= _lib.ROTARY_MAX_AXES or min(pairs) < 0 or sum(pairs) != rot // 2:
            raise ValueError(f"sections must be 1 to {_lib.ROTARY_MAX_AXES} counts that sum to rot / 2")
        kind, factor, original, fast, slow = _lib.SCALING_NONE, 1.0, 1.0, 32.0, 1.0
        if scaling is not None:
            name, *rest = scaling
            if name not in SCALINGS or len(rest) < 1 or len(rest) > (4 if name == "yarn" else 1):
                raise ValueError(f"unknown scaling {scaling!r}")
            kind, factor = SCALINGS[name], float(rest[0])
            if name == "yarn":
                if len(rest) < 2:
                    raise ValueError("yarn needs the original length")
                original = float(rest[1])
                fast, slow = float(rest[2]) if len(rest) > 2 else fast, float(rest[3]) if len(rest) > 3 else slow
        freq, axis = (ctypes.c_uint64 * (rot // 2))(), (ctypes.c_int32 * (rot // 2))()
        g = ctypes.c_float(1.0)
        _check(_lib.lib().solattn_rotary_frequencies(rot, axes, (ctypes.c_int * axes)(*pairs), float(theta), kind, factor,
                                                     original, fast, slow, freq, axis, ctypes.byref(g)),
               "solattn_rotary_frequencies")
        if frequencies is not None:
            values = [float(f) for f in frequencies]
            if len(values) != rot // 2 or not all(math.isfinite(f) for f in values):
                raise ValueError("frequencies must be rot / 2 finite values")
            for i, f in enumerate(values):
                freq[i] = int(round(math.ldexp(math.fmod(f / (2 * math.pi), 1.0), 64))) % (1 << 64)
        self.rot, self.layout, self.axes = rot, layout, axes
        self.gain = float(g.value) if gain is None else float(gain)
        if not math.isfinite(self.gain):
            raise ValueError("gain must be finite")
        device = torch.device("cuda" if device is None else device)
        signed = [f - (1 << 64) if f >= 1 << 63 else f for f in freq]
        self.freq = torch.tensor(signed, dtype=torch.int64).to(device)  # the 64-bit words of solattn_rotary_t.freq
        self.axis = torch.tensor(list(axis), dtype=torch.int32).to(device)

    def _struct(self, positions, B: int, N: int, like: torch.Tensor):
        """solattn_rotary_t for int32 positions [N], [B, N] (one axis) or [N, axes], [B, N, axes]."""
        _same_device(like, self.freq, positions)
        shape = tuple(positions.shape)
        tail = () if self.axes == 1 else (self.axes,)
        if positions.dtype != torch.int32 or shape not in ((N, *tail), (B, N, *tail)):
            raise ValueError("positions must be int32 [N] or [B, N], with a last dimension of the axes when several")
        batched = positions.dim() - len(tail) == 2
        st = positions.stride()
        if tail and st[-1] != 1:
            raise ValueError("the axes of a position must be adjacent")
        token = st[1 if batched else 0]
        if N > 1 and token < 1:
            raise ValueError("positions must not repeat one token's (expand() along N)")
        return _lib.RotaryStruct(self.rot, LAYOUTS[self.layout], self.axes, self.gain, self.freq.data_ptr(),
                                 self.axis.data_ptr(), positions.data_ptr(), st[0] if batched and B > 1 else 0,
                                 token if N > 1 else 0)


def _check_rows(x, d=None):
    if not (x.is_cuda and x.dim() == 4 and (x.shape[-1] <= 1 or x.stride(-1) == 1)):
        raise ValueError("expected CUDA [B, H, N, d] tensors with contiguous d")


def rotary(q, k, rope: Rotary, positions, inverse: bool = False, out=None):
    """q [B, H, N, d] and k [B, H_kv, N, d] (or None) turned by their tokens' positions, in one launch; bf16, fp16 or
    fp32, any strides with a contiguous d. Returns (q', k'). out: a pair of tensors to write (q and k themselves for in
    place). inverse turns back: the gradient of q, k from the gradient of q', k'."""
    _check_rows(q)
    dtype = _dtype(q, fp32=True)
    B, H, N, d = _shape(q)
    if k is not None:
        _check_rows(k)
        if k.dtype != q.dtype or (k.shape[0], k.shape[2], k.shape[3]) != (B, N, d):
            raise ValueError("k must have q's type, batch, tokens and d")
    q_out, k_out = out if out is not None else (torch.empty_like(q), None if k is None else torch.empty_like(k))
    for x, y in ((q, q_out), (k, k_out)):
        if x is None:
            continue
        _check_rows(y)
        if y.shape != x.shape or y.dtype != x.dtype:
            raise ValueError("out must have the inputs' shapes and type")
    _same_device(q, k, q_out, k_out)
    st = rope._struct(positions, B, N, q)
    strides = [None if x is None else _tensor_strides(x) for x in (q, k, q_out, k_out)]
    with _current(q):
        _check(_lib.lib().solattn_rotary(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), dtype, B, H,
                                         0 if k is None else int(k.shape[1]), N, d, *strides, st, int(inverse),
                                         _stream_on(q)), "solattn_rotary")
    return q_out, k_out


def rotary_pool(q, k, v, rope: Rotary, positions, out=None, stats: PooledStats | None = None):
    """rotary() of bf16 q and k and pool() of the result with v, in one pass over them: returns (q', k', stats) for
    forward(q', k', v, stats, ...). The means are those of the rotated values before their rounding. The whole head is
    rotated (rope.rot == d). q and k share v's strides or have strides of their own layout; out as in rotary()."""
    _check_inputs(q, k, v)
    B, H, N, d = _shape(q)
    q_out, k_out = out if out is not None else (torch.empty_like(q), torch.empty_like(k))
    _check_inputs(q_out, k_out)
    if q_out.shape != q.shape:
        raise ValueError("out must have the inputs' shape")
    stats = _pooled_stats(q, stats)
    _same_device(q, k, v, q_out, k_out, stats.buffer)
    st = rope._struct(positions, B, N, q)
    si, so = _strides(q), _strides(q_out)
    with _current(q):
        _check(_lib.lib().solattn_rotary_pool(_ptr(q), _ptr(k), _ptr(v), _ptr(q_out), _ptr(k_out), B, H, N, d, si, so, st,
                                              ctypes.byref(stats.struct), _stream_on(q)), "solattn_rotary_pool")
    return q_out, k_out, stats
