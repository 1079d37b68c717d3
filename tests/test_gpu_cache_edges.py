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


def _cache_of(k, v, seed):
    """A cache that holds k and v [heads, n, d] (fp32) in scattered pages, and its table; scales by the append's rule."""
    H, n, d = k.shape
    columns = (n + 63) // 64
    c = sa.Cache.empty(columns + 2, H, d)
    t = torch.randperm(columns + 2, generator=_gen(seed))[:columns].view(1, columns).to(torch.int32).cuda()
    sa.cache_append(c, k[None].cuda(), v[None].cuda(), t, _i32([0]))
    return c, t


def _held(x8, scale, t, h, n):
    """fp64 [n, d] of what head h of the cache holds."""
    p = t[0].long().cpu()
    return (x8.cpu()[p, h].double() * scale.cpu()[p, h].double()[:, None, None]).flatten(0, 1)[:n]


COPIES = 222  # sequences with the same pages and queries: enough of them that no key axis is split


def _attend_and_check(q, c, t, n, causal):
    for copies in (COPIES, 1):
        _attend_copies(q, c, t, n, causal, copies)


def _attend_copies(q, c, t, n, causal, copies):
    """A call of many equal sequences: the same bits for each, and 64-bit attention on the held values. The bounds are
    those of the weights' rounding (2^-11 of a weight), of scores (delta = 2^-18 sum |q||k| scale), of sums and
    exponentials (2^-15); and what a weight below fp16's normal range loses, 2^-25 in units where the row's largest is
    2^4 at least. Those units hold weight times value scale, each scale within 2^6 of the unit that follows them, so of
    every value that a row sees at most 2^-25 2^-4 2^6 2^6 |v|."""
    _, H, N, d = q.shape
    out, lse = sa.cache_attention(q.expand(copies, H, N, d), c, t.repeat(copies, 1), _i32([n] * copies), causal=causal,
                                  out=torch.empty((copies, H, N, d), dtype=q.dtype, device="cuda"))
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    eps = torch.finfo(q.dtype).eps
    for h in range(H):
        j = h // (H // c.heads)
        k, v = _held(c.k, c.k_scale, t, j, n), _held(c.v, c.v_scale, t, j, n)
        o, l, mag, size = ref.attend(q[0, h].cpu(), k, v, causal, N, d ** -0.5)
        total = v.abs().cumsum(0)
        total = torch.stack([total[max(0, n - N + i) if causal else n - 1] for i in range(N)])
        delta = 2.0 ** -18 * size[:, None]
        tol = (2.0 ** -11 + 2.0 ** -15 + 2 * delta) * mag + 2.0 ** -17 * total + eps / 2 * 1.01 * o.abs()
        err = (out[0, h].cpu().double() - o).abs()
        assert (err <= tol).all(), (h, float((err / tol.clamp(min=1e-30)).max()))
        e2 = (lse[0, h].cpu().double() - l).abs()
        assert (e2 <= delta[:, 0] + 2.0 ** -15 + 2.0 ** -22 * l.abs()).all()


OUTLIERS = [
    # tokens, (token, column, value) of the outliers
    (128, [(127, 5, 1e9)]),                        # the second page's last token
    (500, [(200, 0, 1e9), (201, 63, -3e8)]),       # pages of ordinary size before and behind
    (700, [(0, 1, 1e12), (699, 2, 1e12)]),         # the first and the last page
    (900, [(64 * i + 9, i, 10.0 ** (i % 5 * 3)) for i in range(14)]),  # every page another size
    (4500, [(64 * i + 7, i % 60, 1e9) for i in (0, 29, 31, 32, 33, 34, 40, 62, 63, 64, 66, 70)]),  # around 32 and 64 pages
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [2, 60, 140])
@pytest.mark.parametrize("n,outliers", OUTLIERS)
def test_one_large_value_leaves_other_tokens_and_columns_alone(n, outliers, N, d):
    """Values with an outlier in one column: its page's scale rises until the page's other values are 0, and the rows in
    front of it and every other column still have the other pages' values to full accuracy."""
    H, N = 2, min(N, n)
    k, v = (torch.randn((H, n, d), generator=_gen(i + n)) for i in range(2))
    for token, column, value in outliers:
        v[:, token, column] = value
    c, t = _cache_of(k, v, seed=n)
    q = torch.randn((1, 2 * H, N, d), generator=_gen(N)).to(torch.bfloat16).cuda()
    for causal in (True, False):
        _attend_and_check(q, c, t, n, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 30, 100])
def test_value_scales_over_the_whole_range(N, d):
    """Pages' value scales from 2^-32 to 2^32 in any order, zero pages among them; a whole column that only the smallest
    page fills comes out accurately."""
    n, H = 64 * 9, 1
    k, v = (torch.randn((H, n, d), generator=_gen(i + 77)) for i in range(2))
    exponents = [-32, 32, -32, 0, 31, -9, 12, -20, 4]
    v = v.view(H, 9, 64, d)
    for i, e in enumerate(exponents):
        v[:, i] = (v[:, i] / v[:, i].abs().amax()) * 440.0 * 2.0 ** e
        v[:, i, :, 7] *= i == 2
    v[:, 6] = 0
    c, t = _cache_of(k, v.view(H, n, d), seed=3)
    held = c.v_scale[t[0].long()]
    assert float(held.min()) == 2.0 ** -32 and float(held.max()) == 2.0 ** 32
    q = torch.randn((1, 2, N, d), generator=_gen(N)).to(torch.bfloat16).cuda()
    for causal in (True, False):
        _attend_and_check(q, c, t, n, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 64, 200])
def test_expired_waits_of_short_parts(n, d):
    """Parts of at most four pages, all of whose copies are on their way before a wait is due: where the first page never
    comes, every block ends with its other copies landed, and the next call gives its bits, time after time."""
    B, H = 90, 2
    k, v = (torch.randn((H, n, d), generator=_gen(i + n)) for i in range(2))
    c, t = _cache_of(k, v, seed=n)
    t = t.repeat(B, 1)
    q = torch.randn((B, H, 2, d), generator=_gen(4)).to(torch.bfloat16).cuda()
    lengths = _i32([n] * B)
    ws = sa.cache_workspace(q, c, t)
    want, want_lse = sa.cache_attention(q, c, t, lengths, ws=ws)
    lib = _lib.lib()
    for _ in range(3):
        assert lib.solattn_test_set_hook(0, 20_000_000) == 0
        try:
            sa.cache_attention(q, c, t, lengths, ws=ws)
            assert sa.status(ws) == _lib.ERR_TIMEOUT
        finally:
            assert lib.solattn_test_set_hook(-1, 2_000_000_000) == 0
        ws[:_lib.WORKSPACE_BYTES].zero_()
        out, lse = sa.cache_attention(q, c, t, lengths, ws=ws)
        assert sa.status(ws) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("N", [1, 20, 150])
def test_scale_that_is_no_number(N, which):
    """A page whose scale is NaN gives NaN in the rows that see one of its tokens, in either kernel, and leaves the other
    rows' bits alone."""
    n, H, d = 320, 1, 128
    k, v = (torch.randn((H, n, d), generator=_gen(i + 5)) for i in range(2))
    c, t = _cache_of(k, v, seed=8)
    q = torch.randn((1, 2, N, d), generator=_gen(N)).to(torch.bfloat16).cuda()
    for causal in (True, False):
        clean, clean_lse = sa.cache_attention(q, c, t, _i32([n]), causal=causal)
        page = int(t[0, 4])  # tokens 256 .. 319
        old = float(getattr(c, which)[page, 0])
        getattr(c, which)[page, 0] = math.nan
        out, lse = sa.cache_attention(q, c, t, _i32([n]), causal=causal)
        getattr(c, which)[page, 0] = old
        blind = max(0, N - 64) if causal else 0
        assert torch.equal(out[:, :, :blind], clean[:, :, :blind]) and torch.equal(lse[:, :, :blind], clean_lse[:, :, :blind])
        assert torch.isnan(out[:, :, blind:]).all() and torch.isnan(lse[:, :, blind:]).all()
