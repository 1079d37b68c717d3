"""The cache attention's tests again, through each of its two kernels whatever the sizes: the test-hook build takes the
named one where the product library would take the one that it estimates to be faster."""
import pytest

from block_sparse_attention_cov_b200 import _cache, _lib
from block_sparse_attention_cov_b200.build import build
from hooklib import hooks_lib
from test_gpu_cache import (  # noqa: F401
    test_attention_against_formula, test_attention_extreme_queries_and_scales,
    test_attention_long_table_short_sequences, test_attention_not_finite, test_attention_of_many_sequences, test_attention_of_zero_queries_and_zero_values,
    test_attention_strides_streams_and_repeats, test_bad_pages_lengths_and_counts_are_reported_and_touch_nothing,
    test_every_e4m3_value_is_read_exactly, test_rows_that_see_nothing_at_any_value_scale,
    test_together_as_a_decoder_uses_them)
from test_gpu_cache_use import (  # noqa: F401
    test_expired_wait_reports_timeout_and_next_call_succeeds, test_two_calls_at_once)

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 2], ids=["few", "many"], autouse=True)
def _kernel(request, monkeypatch):
    import torch
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
