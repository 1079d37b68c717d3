"""Refusals by the binding for CUDA tensors, made as shapes and strides only (no device, no memory): what the kernels could
not read or write in bounds is refused before its address is asked for."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import block_sparse_attention_cov_b200 as sa

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
