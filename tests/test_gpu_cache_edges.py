"""Corners of attention over the 8-bit cache, through the kernel that the estimates choose and through each of the two."""
import math

import pytest
import torch

import block_sparse_attention_cov_b200 as sa
import ops_ref as ref
from block_sparse_attention_cov_b200 import _cache, _lib
from block_sparse_attention_cov_b200.build import build
from hooklib import hooks_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[0, 1, 2], ids=["chosen", "few", "many"], autouse=True)
def _kernel(request, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build()
    lib = hooks_lib()
    monkeypatch.setattr(_lib, "_lib", lib)
    lib.solattn_test_set_cache_kernel(request.param)
    _cache._workspace_bytes.cache_clear()
    yield
    lib.solattn_test_set_cache_kernel(0)
    _cache._workspace_bytes.cache_clear()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tiles_that_see_no_page(d, dtype):
    """Whole tiles of queries without a key, and others with some, in one unsplit call: 0 and -inf every time, and what a
    query wrote into the tile on its way never shows."""
    lengths = [0, 1, 64, 0, 20, 0]
    B, H, Hk, N = len(lengths), 4, 2, 512
    c = sa.Cache.empty(B, Hk, d)
    c.k.view(torch.uint8).random_(0, 0x70, generator=torch.Generator("cuda").manual_seed(1))
    c.v.view(torch.uint8).random_(0x30, 0x70, generator=torch.Generator("cuda").manual_seed(2))
    c.k_scale.fill_(0.01), c.v_scale.fill_(0.25)
    t = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    q = (1e4 + 1e4 * torch.rand((B, H, N, d), generator=_gen(3))).to(dtype).cuda()
    ws = sa.cache_workspace(q, c, t)
    lens = _i32(lengths)
    for causal in (True, False):
        for _ in range(40):
            out, lse = sa.cache_attention(q, c, t, lens, causal=causal, ws=ws)
            for b, n in enumerate(lengths):
                blind = N - n if causal else (N if n == 0 else 0)
                assert (out[b, :, :blind] == 0).all() and (lse[b, :, :blind] == -math.inf).all()
                assert (out[b, :, blind:] > 0).all() and torch.isfinite(lse[b, :, blind:]).all()
    assert sa.status(ws) == 0
