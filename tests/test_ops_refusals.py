"""Refusals of the operators around attention (CPU: every call below fails validation before it touches a device), and
the rotary frequencies, which the host computes."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_cov_b200 as sa
import ops_ref as ref
from block_sparse_attention_cov_b200 import _lib
from block_sparse_attention_cov_b200.build import build

P = ctypes.c_void_p
FAKE = P(0x7F0000000000)
ODD = P(0x7F0000000008)   # 8-byte aligned only
OFF1 = P(0x7F0000000001)
OFF2 = P(0x7F0000000002)
S = _lib.StridesStruct


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


def _rope(**kw):
    f = dict(rot=64, layout=1, axes=1, gain=1.0, freq=0x7F0000000000, axis=None, positions=0x7F0000000000,
             position_batch=0, position_token=0)
    f.update(kw)
    return _lib.RotaryStruct(*[f[n] for n, _ in _lib.RotaryStruct._fields_])


def _rotary(L, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, dtype=0, B=1, H=2, Hk=1, N=8, d=64, st=(None,) * 4, rope="default"):
    rope = _rope() if rope == "default" else rope
    return L.solattn_rotary(q, k, qo, ko, dtype, B, H, Hk, N, d, *st, rope, 0, None)


def test_rotary_refusals(L):
    A, U, G = _lib.ERR_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_ALIGN
    assert _rotary(L, q=None) == A and _rotary(L, qo=None) == A and _rotary(L, ko=None) == A
    assert _rotary(L, B=0) == A and _rotary(L, N=-1) == A and _rotary(L, H=0) == A and _rotary(L, Hk=0) == A
    assert _rotary(L, d=0) == A and _rotary(L, rope=None) == A
    assert _rotary(L, dtype=3) == U and _rotary(L, dtype=-1) == U
    assert _rotary(L, d=1026) == U
    assert _rotary(L, B=1 << 12, N=1 << 13) == U     # B N d beyond 2^31
    assert _rotary(L, H=65536) == U
    for bad in (dict(rot=0), dict(rot=3), dict(rot=66), dict(rot=-2), dict(layout=2), dict(axes=0), dict(axes=5),
                dict(axes=3), dict(gain=math.nan), dict(gain=math.inf), dict(freq=None), dict(positions=None),
                dict(position_batch=-1), dict(position_token=-4)):
        assert _rotary(L, rope=_rope(**bad)) == A, bad
    assert _rotary(L, rope=_rope(freq=0x7F0000000004)) == G
    assert _rotary(L, rope=_rope(positions=0x7F0000000002)) == G
    assert _rotary(L, q=OFF1) == G and _rotary(L, ko=OFF1) == G
    assert _rotary(L, q=OFF2, dtype=2) == G
    bad = S(-1, 64, 128)
    for at in range(4):
        st = [None] * 4
        st[at] = bad
        assert _rotary(L, st=st) == A
    # outputs whose rows overlap
    assert _rotary(L, st=(None, None, S(1024, 512, 32), None)) == A
    assert _rotary(L, st=(None, None, S(1024, 0, 64), None)) == A


def test_rotary_pool_refusals(L):
    def call(q=FAKE, qo=FAKE, H=2, N=128, d=64, st=None, so=None, rope=None, pooled="default", B=1):
        p = _lib.PooledStruct(*[0x7F0000000000] * 7) if pooled == "default" else pooled
        return L.solattn_rotary_pool(q, FAKE, FAKE, qo, FAKE, B, H, N, d, st, so, rope or _rope(), p, None)
    A, U, G = _lib.ERR_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_ALIGN
    assert call(q=None) == A and call(qo=None) == A and call(N=0) == A and call(pooled=None) == A
    assert call(q=ODD) == G and call(qo=ODD) == G
    assert call(d=96) == U and call(N=_lib.MAX_TOKENS + 1) == U
    assert call(rope=_rope(rot=32)) == U          # the whole head or rotary() and pool()
    assert call(rope=_rope(rot=64), d=128) == U
    assert call(H=65536, N=1) == U
    assert call(st=S(0, 8, 60)) == A and call(so=S(128 * 64, 0, 64)) == A and call(so=S(8, 4, 64)) == A
    assert call(pooled=_lib.PooledStruct(*[0x7F0000000000] * 6, None)) == A


def _cache(**kw):
    f = dict(k=FAKE.value, v=FAKE.value, k_scale=FAKE.value, v_scale=FAKE.value, pages=4, heads=2, d=64, page_stride=0,
             scale_stride=0)
    f.update(kw)
    return _lib.CacheStruct(*[f[n] for n, _ in _lib.CacheStruct._fields_])


BAD_CACHES = [dict(k=None), dict(v_scale=None), dict(pages=0), dict(heads=0), dict(page_stride=-16),
              dict(page_stride=64 * 64), dict(page_stride=2 * 64 * 64 + 8), dict(scale_stride=1), dict(scale_stride=-2)]


def test_append_refusals(L):
    def call(k=FAKE, v=FAKE, dtype=0, B=1, N=3, st=None, cache="default", table=FAKE, columns=2, ts=0, lengths=FAKE,
             counts=None, ws=None, wsb=0):
        c = _cache() if cache == "default" else cache
        return L.solattn_cache_append(k, v, dtype, B, N, st, c, table, columns, ts, lengths, counts, ws, wsb, None)
    A, U, G = _lib.ERR_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_ALIGN
    assert call(k=None) == A and call(v=None) == A and call(B=0) == A and call(N=0) == A and call(cache=None) == A
    assert call(table=None) == A and call(lengths=None) == A and call(columns=0) == A and call(ts=1) == A and call(ts=-2) == A
    for bad in BAD_CACHES:
        assert call(cache=_cache(**bad)) == A, bad
    assert call(cache=_cache(d=96)) == U and call(dtype=7) == U and call(columns=(1 << 22) + 1) == U and call(B=32768) == U
    assert call(k=ODD) == G and call(cache=_cache(k=0x7F0000000008)) == G and call(cache=_cache(k_scale=0x7F0000000002)) == G
    assert call(lengths=OFF2) == G and call(counts=OFF2) == G and call(table=OFF2) == G and call(ws=ODD, wsb=256) == G
    assert call(st=S(1024, 512, 60)) == A and call(st=S(-8, 512, 64)) == A
    assert call(ws=FAKE, wsb=255) == _lib.ERR_WORKSPACE


def test_attention_refusals(L):
    def call(q=FAKE, dtype=0, B=1, H=4, N=1, d=64, st=None, cache="default", table=FAKE, columns=2, ts=0, lengths=FAKE,
             counts=None, scale=0.0, out=FAKE, so=None, lse=None, ws=FAKE, wsb=1 << 30):
        c = _cache() if cache == "default" else cache
        return L.solattn_cache_attention(q, dtype, B, H, N, d, st, c, table, columns, ts, lengths, counts, 1, scale, out,
                                         so, lse, ws, wsb, None)
    A, U, G, W = _lib.ERR_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_ALIGN, _lib.ERR_WORKSPACE
    assert call(q=None) == A and call(out=None) == A and call(cache=None) == A and call(table=None) == A
    assert call(lengths=None) == A and call(B=0) == A and call(N=0) == A and call(H=0) == A and call(columns=0) == A
    assert call(H=3) == A                                    # no multiple of the cache's heads
    assert call(d=128) == A                                  # the cache's d is 64
    assert call(d=96, cache=_cache(d=96)) == U and call(dtype=2) == U and call(columns=(1 << 22) + 1) == U
    assert call(B=65536) == U and call(H=16386) == U and call(B=1 << 15, H=1 << 14, N=4) == U
    for bad in BAD_CACHES:
        assert call(cache=_cache(**bad)) in (A,), bad
    assert call(scale=-1.0) == A and call(scale=math.nan) == A and call(scale=math.inf) == A
    assert call(q=ODD) == G and call(out=ODD) == G and call(lse=OFF2) == G and call(ws=ODD) == G and call(counts=OFF2) == G
    assert call(st=S(1024, 64, 4)) == A and call(so=S(1024, 0, 64)) == A and call(so=S(1024, 64, 32), N=2) == A
    n = ctypes.c_size_t()
    assert L.solattn_cache_workspace_bytes(1, 4, 1, 64, 2, 2, ctypes.byref(n)) == _lib.OK
    assert call(ws=None) == W and call(wsb=n.value - 1) == W
    assert L.solattn_cache_workspace_bytes(1, 4, 1, 64, 2, 2, None) == A
    assert L.solattn_cache_workspace_bytes(1, 4, 1, 64, 3, 2, ctypes.byref(n)) == A


def test_workspace_covers_every_split(L):
    """The size follows the plan: the status block alone where the key axis is not split, and room for d + 2 floats per
    row and part else."""
    n = ctypes.c_size_t()
    for B, H, N, d, Hk, cols in ((64, 8, 1, 128, 8, 1), (1, 8, 1, 128, 8, 1024), (1, 1, 700, 64, 1, 4096), (8, 40, 4000, 128, 8, 60)):
        assert L.solattn_cache_workspace_bytes(B, H, N, d, Hk, cols, ctypes.byref(n)) == _lib.OK
        parts, rest = divmod(n.value - 256, B * H * N * (d + 2) * 4)
        assert rest == 0 and (parts == 0 or 2 <= parts <= cols)


@pytest.mark.parametrize("pairs,scaling", [((64,), None), ((22, 21, 21), None), ((32,), ("linear", 4.0)), ((16, 8), ("ntk", 8.0)),
                                           ((64,), ("yarn", 8.0, 32768)), ((24,), ("yarn", 2.0, 100, 20.0, 0.5))])
def test_rotary_frequencies(L, pairs, scaling):
    want, axis, gain = ref.frequencies(pairs, 10000.0, scaling)
    n = sum(pairs)
    f, a, g = (ctypes.c_uint64 * n)(), (ctypes.c_int32 * n)(), ctypes.c_float()
    kind = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}[scaling and scaling[0]]
    rest = list(scaling[2:]) if scaling and kind == 3 else []
    original, fast, slow = rest + [1.0, 32.0, 1.0][len(rest):]
    rc = L.solattn_rotary_frequencies(2 * n, len(pairs), (ctypes.c_int * len(pairs))(*pairs), 10000.0, kind,
                                      scaling[1] if scaling else 1.0, original, fast, slow, f, a, ctypes.byref(g))
    assert rc == _lib.OK and list(a) == axis and g.value == pytest.approx(gain, rel=1e-7)
    for x, y in zip(f, want):
        assert x / 2.0 ** 64 * 2 * math.pi == pytest.approx(y, rel=1e-14)


def test_rotary_frequencies_refusals(L):
    f, a, g = (ctypes.c_uint64 * 64)(), (ctypes.c_int32 * 64)(), ctypes.c_float()

    def call(rot=64, axes=1, pairs=None, theta=1e4, kind=0, factor=2.0, original=10.0, fast=32.0, slow=1.0, freq=f, ax=a):
        p = None if pairs is None else (ctypes.c_int * len(pairs))(*pairs)
        return L.solattn_rotary_frequencies(rot, axes, p, theta, kind, factor, original, fast, slow, freq, ax, ctypes.byref(g))
    assert call() == _lib.OK and call(ax=None) == _lib.OK
    for bad in (dict(rot=0), dict(rot=7), dict(axes=0), dict(axes=5, pairs=[1] * 5), dict(axes=2), dict(axes=2, pairs=[16, 15]),
                dict(axes=2, pairs=[33, -1]), dict(axes=2, pairs=[16, 16], ax=None), dict(theta=1.0), dict(theta=math.nan),
                dict(theta=math.inf), dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=1, factor=math.nan),
                dict(kind=3, original=0.0), dict(kind=3, fast=1.0, slow=1.0), dict(kind=3, slow=0.0), dict(freq=None),
                dict(kind=2, axes=2, pairs=[31, 1])):
        assert call(**bad) == _lib.ERR_ARG, bad


def test_python_refusals_without_a_device(L):
    """CPU tensors, wrong types and shapes are refused by the binding."""
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sa.rotary(x, None, None, None)
    with pytest.raises(ValueError):
        sa.rotary_pool(x, x, x, None, None)
    with pytest.raises(ValueError):
        sa.cache_attention(x, None, None, None)
    z8 = torch.zeros((2, 1, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        sa.Cache(z8, z8, torch.zeros(2, 1), torch.zeros(2, 1))
    with pytest.raises(ValueError):
        sa.Rotary(63)
    with pytest.raises(ValueError):
        sa.Rotary(64, layout="diagonal")
    with pytest.raises(ValueError):
        sa.Rotary(64, sections=(10, 10))
    with pytest.raises(ValueError):
        sa.Rotary(64, scaling=("yarn", 2.0))
    with pytest.raises(ValueError):
        sa.Rotary(64, scaling=("other", 2.0))
    with pytest.raises(sa.SolAttnError):
        sa.Rotary(64, theta=0.5)
