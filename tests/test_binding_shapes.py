"""Refusals by the binding for CUDA tensors, made as shapes and strides only (no device, no memory): what the kernels could
not read or write in bounds is refused before its address is asked for."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import block_sparse_attention_cov_b200 as sa
from block_sparse_attention_cov_b200 import _lib

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
