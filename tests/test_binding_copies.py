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
