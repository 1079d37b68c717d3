"""Refusals by the binding for CUDA tensors, made as shapes and strides only (no device, no memory): what the kernels could
not read or write in bounds is refused before its address is asked for."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import block_sparse_attention_cov_b200 as sa
from block_sparse_attention_cov_b200 import _lib
from block_sparse_attention_cov_b200.build import build

E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _shapes_only():
    with FakeTensorMode():
        yield


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def test_cache_of_one_page_or_scale_repeated():
    """expand() along the pages has step 0, which the C call would take for contiguous memory."""
    k, s = _empty(4, 2, 64, 64, dtype=E4M3), _empty(4, 2)
    one, scale = _empty(1, 2, 64, 64, dtype=E4M3).expand(4, 2, 64, 64), _empty(1, 2).expand(4, 2)
    for keys, scales in ((one, s), (k, scale), (one, scale), (k, _empty(2).expand(4, 2))):
        with pytest.raises(ValueError, match="pages"):
            sa.Cache(keys, keys, scales, scales)


@pytest.mark.parametrize("call", ["pool", "forward", "rotary", "rotary_out", "rotary_pool", "rotary_pool_out"])
def test_tensors_of_one_row_repeated(call, monkeypatch):
    """expand() along batch, heads and tokens leaves three steps of 0, which the C calls take for contiguous memory."""
    class Library:
        def __getattr__(self, name):
            def reached(*args):
                raise AssertionError(f"{name} was called")
            return reached

    monkeypatch.setattr(_lib, "lib", Library)
    whole = _empty(2, 3, 70, 64, dtype=torch.bfloat16)
    row = _empty(1, 1, 1, 64, dtype=torch.bfloat16).expand(2, 3, 70, 64)
    assert row.stride() == (0, 0, 0, 1)
    stats = sa.PooledStats(whole, None, (2, 3, 70, 64))
    rope = sa.Rotary.__new__(sa.Rotary)
    rope.freq = rope.axis = whole
    rope._struct = lambda *a: None
    with pytest.raises(ValueError, match="repeated row"):
        if call == "pool":
            sa.pool(row, row, row, stats)
        elif call == "forward":
            sa.forward(row, row, row, stats, rule="topk", topk=1, out=row, ws=whole)
        elif call == "rotary":
            sa.rotary(row, None, rope, whole)
        elif call == "rotary_out":
            sa.rotary(whole, None, rope, whole, out=(row, None))
        elif call == "rotary_pool":
            sa.rotary_pool(row, row, row, rope, whole, out=(whole, whole), stats=stats)
        else:
            sa.rotary_pool(whole, whole, whole, rope, whole, out=(row, row), stats=stats)


@pytest.mark.parametrize("scale", [1e-50, 1e-46, 3e38, 1e39, 0.0, -1.0, float("nan"), float("inf")])
def test_softmax_scales_that_are_none(scale):
    """The C call takes the scale in fp32, where a tiny one becomes 0 (its word for the default) and a huge one infinite,
    there or when it is brought to base 2."""
    q, i = _empty(1, 2, 1, 64, dtype=torch.bfloat16), _empty(1, dtype=torch.int32)
    cache = type("C", (), {"d": 64, "heads": 2, "k": q})()
    with pytest.raises(ValueError, match="scale"):
        sa.cache_attention(q, cache, _empty(1, 1, dtype=torch.int32), i, scale=scale)


def test_softmax_scale_beyond_base_two_is_refused_by_the_library():
    build()
    fake, st = ctypes.c_void_p(0x7F0000000000), _lib.CacheStruct(*[0x7F0000000000] * 4, 4, 2, 64, 0, 0)
    for scale, want in ((2.5e38, _lib.ERR_ARG), (float("inf"), _lib.ERR_ARG), (-1e-30, _lib.ERR_ARG)):
        assert _lib.lib().solattn_cache_attention(fake, 0, 1, 4, 1, 64, None, st, fake, 2, 0, fake, None, 1, scale, fake, None,
                                                  None, fake, 1 << 30, None) == want
