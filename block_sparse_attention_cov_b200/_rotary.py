"""Rotary positions on queries and keys (solattn_rotary, solattn_rotary_pool)."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from . import (PooledStats, _at, _call, _check, _check_inputs, _device_index, _dtype, _pooled_stats, _strides_struct,
               _tensor_strides)

__all__ = ["Rotary", "rotary", "rotary_pool"]

LAYOUTS = {"interleaved": _lib.ROTARY_INTERLEAVED, "half": _lib.ROTARY_HALF}
SCALINGS = {"linear": _lib.SCALING_LINEAR, "ntk": _lib.SCALING_NTK, "yarn": _lib.SCALING_YARN}


class Rotary:
    """The frequencies of a rotary embedding, on the device, made once and used by every call.

    rot: rotated leading elements of a head (even). layout: "half" (element p pairs with p + rot/2) or "interleaved"
    (2p with 2p + 1). sections: rotated pairs of each position axis (for video, t, h and w), each with frequencies
    theta^(-i / n) of its own; None: one axis. scaling: None, ("linear", factor), ("ntk", factor) or
    ("yarn", factor, original_length[, fast, slow]), whose ramp is linear in a pair's turns within the original length
    (for one linear in the pair's index give the frequencies and the gain). frequencies: rot / 2 values in radians per position that replace
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
        self._layout = LAYOUTS[layout]

    def _struct(self, positions, B: int, N: int):
        """solattn_rotary_t for int32 positions [N], [B, N] (one axis) or [N, axes], [B, N, axes]."""
        shape, st = positions.shape, positions.stride()
        several = self.axes > 1
        lead = len(shape) - several
        if positions.dtype != torch.int32 or not 1 <= lead <= 2 or shape[lead - 1] != N or (lead == 2 and shape[0] != B) \
                or (several and (shape[-1] != self.axes or st[-1] != 1)):
            raise ValueError("positions must be int32 [N] or [B, N], with a last, contiguous dimension of the axes where "
                             "there are several")
        token = st[lead - 1] if N > 1 else 0
        if N > 1 and token < 1:
            raise ValueError("positions must not be one token's repeated (expand() along N)")
        # the addresses as they are now: a copy of the object, or one whose tables moved, has other ones
        return _lib.RotaryStruct(self.rot, self._layout, self.axes, self.gain, self.freq.data_ptr(), self.axis.data_ptr(),
                                 positions.data_ptr(), st[0] if lead == 2 and B > 1 else 0, token)


def _outputs(q, k, out):
    if out is None:
        return torch.empty_like(q), None if k is None else torch.empty_like(k)
    for x, y in zip((q, k), out):
        if x is not None and (y.shape != x.shape or y.dtype != x.dtype or y.stride(-1) != 1):
            raise ValueError("out must have the inputs' shapes and type, and a contiguous d")
    return out[0], None if k is None else out[1]


def rotary(q, k, rope: Rotary, positions, inverse: bool = False, out=None):
    """q [B, H, N, d] and k [B, H_kv, N, d] (or None) turned by their tokens' positions, in one launch; bf16, fp16 or
    fp32, any strides with a contiguous d. Returns (q', k'). out: a pair of tensors to write (q and k themselves for in
    place). inverse turns back: the gradient of q, k from the gradient of q', k'."""
    if q.dim() != 4 or q.stride(3) != 1 or (k is not None and (k.dim() != 4 or k.stride(3) != 1)):
        raise ValueError("expected [B, H, N, d] tensors with contiguous d")
    dtype = _dtype(q)
    B, H, N, d = q.shape
    Hk = 0
    if k is not None:
        Bk, Hk, Nk, dk = k.shape
        if k.dtype != q.dtype or (Bk, Nk, dk) != (B, N, d):
            raise ValueError("k must have q's type, batch, tokens and d")
    if q.get_device() < 0:
        raise ValueError("expected CUDA tensors")
    q_out, k_out = _outputs(q, k, out)
    dev = _device_index(q, k, q_out, k_out, rope.freq, rope.axis, positions)
    _call("solattn_rotary", _lib.lib().solattn_rotary, dev, q.data_ptr(), _at(k), q_out.data_ptr(), _at(k_out), dtype, B, H,
          Hk, N, d, _tensor_strides(q), None if k is None else _tensor_strides(k), _tensor_strides(q_out),
          None if k is None else _tensor_strides(k_out), rope._struct(positions, B, N), 1 if inverse else 0)
    return q_out, k_out


def rotary_pool(q, k, v, rope: Rotary, positions, out=None, stats: PooledStats | None = None):
    """rotary() of bf16 q and k [B, H, N, d] and pool() of the result with v, in one pass over the three: returns
    (q', k', stats) for forward(q', k', v, stats, ...). The means are those of the rotated values before their rounding
    to bf16. The whole head is rotated (rope.rot == d). q, k and v share their strides, and so do the two outputs; out
    as in rotary()."""
    _check_inputs(q, k, v)
    B, H, N, d = q.shape
    q_out, k_out = _outputs(q, k, out)
    if q_out.stride() != k_out.stride():
        raise ValueError("the outputs must share their strides")
    stats = _pooled_stats(q, stats)
    dev = _device_index(q, k, v, q_out, k_out, stats.buffer, rope.freq, rope.axis, positions)
    _call("solattn_rotary_pool", _lib.lib().solattn_rotary_pool, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          q_out.data_ptr(), k_out.data_ptr(), B, H, N, d, _shared_strides(q), _shared_strides(q_out),
          rope._struct(positions, B, N), stats.struct)
    return q_out, k_out, stats


def _shared_strides(t):
    """The strides as they are, for the calls that check every one of them."""
    if t.is_contiguous():
        return None
    strides = t.stride()[:3]
    if not any(strides):
        raise ValueError("a tensor of one repeated row (expand()) is not supported")
    return _strides_struct(*strides)
