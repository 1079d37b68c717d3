"""Objects of the binding that a program copies, pickles or re-targets keep pointing at the memory that they hold."""
import copy
import ctypes
import pickle

import pytest
import torch

import block_sparse_attention_cov_b200 as sa
from block_sparse_attention_cov_b200 import _lib
from block_sparse_attention_cov_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("copied", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))],
                         ids=["copy", "deepcopy", "pickle"])
def test_rotary_copies_point_at_their_own_frequencies(copied):
    rope = sa.Rotary(64, layout="interleaved", sections=(12, 10, 10), device="cpu")
    pos = torch.zeros((5, 3), dtype=torch.int32)
    other = copied(rope)
    assert torch.equal(other.freq, rope.freq) and torch.equal(other.axis, rope.axis)
    for r in (rope, other):
        st = r._struct(pos, 2, 5)
        assert st.freq == r.freq.data_ptr() and st.axis == r.axis.data_ptr()
    rope.freq, rope.axis = rope.freq.clone(), rope.axis.clone()  # a move of the tables to other memory
    st = rope._struct(pos, 2, 5)
    assert st.freq == rope.freq.data_ptr() and st.axis == rope.axis.data_ptr()


def _stats(B, H, N, d, lead=0):
    """PooledStats over CPU memory whose arrays start `lead` bytes into the buffer."""
    n, st = ctypes.c_size_t(0), _lib.PooledStruct()
    buf = torch.empty(sa.pooled_bytes(B, H, N, d) + lead + 256, dtype=torch.uint8)
    at = (buf.data_ptr() + 255) // 256 * 256 + lead
    assert _lib.lib().solattn_pooled_layout(B, H, N, d, at, ctypes.byref(st), ctypes.byref(n)) == 0
    return sa.PooledStats(buf, st, (B, H, N, d))


ARRAYS = ("qbar", "kbar", "vbar", "kmean", "kcov", "kbar16", "vbar16")


def test_pooled_views_follow_struct_and_buffer():
    """A view is the memory that the C calls write: the struct's address, in the buffer held now."""
    B, H, N, d = 2, 3, 200, 64
    stats = _stats(B, H, N, d)
    for turn in range(3):
        for name in ARRAYS:
            v = stats.view(name)
            assert v.data_ptr() == getattr(stats.struct, name) and v.is_contiguous()
            v.fill_(turn + 1)
        assert all((stats.view(name) == turn + 1).all() for name in ARRAYS)
        old = stats.buffer
        other = _stats(B, H, N, d, lead=512 * (turn + 1))
        stats.buffer, stats.struct = other.buffer, other.struct
        assert all(stats.view(name).untyped_storage().data_ptr() == other.buffer.data_ptr() for name in ARRAYS)
        assert not any(v is not stats.buffer and isinstance(v, torch.Tensor)
                       and v.untyped_storage().data_ptr() == old.data_ptr() for v in vars(stats).values())
    assert set(vars(stats)) >= {"buffer", "struct", "shape"} and all(isinstance(k, str) for k in vars(stats))


def test_pooled_views_of_arrays_laid_out_by_the_caller():
    """Arrays in another order than solattn_pooled_layout's."""
    B, H, N, d = 1, 2, 64, 64
    stats = _stats(B, H, N, d)
    stats.struct.qbar, stats.struct.kbar = stats.struct.kbar, stats.struct.qbar
    for name in ARRAYS:
        assert stats.view(name).data_ptr() == getattr(stats.struct, name)


def _cache(monkeypatch, pages=3, heads=2, d=64):
    """A Cache over CPU memory (its check for a device passed over)."""
    from block_sparse_attention_cov_b200 import _cache
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(_cache, "_device_index", lambda *ts: 0)
    k, v = (torch.zeros((pages, heads, 64, d), dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
    return sa.Cache(k, v, torch.ones(pages, heads), torch.ones(pages, heads))


def _points_at_its_own(c):
    return (c.struct.k, c.struct.v, c.struct.k_scale, c.struct.v_scale) == \
        tuple(x.data_ptr() for x in (c.k, c.v, c.k_scale, c.v_scale))


@pytest.mark.parametrize("copied", [copy.copy, copy.deepcopy])
def test_cache_copies_point_at_their_own_pages(copied, monkeypatch):
    c = _cache(monkeypatch)
    other = copied(c)
    assert _points_at_its_own(c) and _points_at_its_own(other)
    assert torch.equal(other.k_scale, c.k_scale) and (other.pages, other.heads, other.d) == (c.pages, c.heads, c.d)


def test_cache_tensors_cannot_be_replaced_under_their_addresses(monkeypatch):
    c = _cache(monkeypatch)
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name).clone())
    assert _points_at_its_own(c)
