"""The 8-bit cache: writing tokens (solattn_cache_append) bit for bit against a plain form, and attention over it
(solattn_cache_attention) against 64-bit softmax attention on the values the cache stands for.

Tolerance of attention. A weight is rounded to fp16 for the value product (2^-11 of itself at most, weights under 2^-30
of the row's largest dropped: 2^-30 L in all, within 2^-16 here); a score is an fp32 sum of d products, off by at most
delta = 2^-18 sum |q||k| scale, which moves a weight by as much and the normaliser too (2 delta); fp32 exponentials, sums
and the join add 2^-16. With A = sum p |v| / sum p:
    |out - exact| <= (2^-11 + 2^-15 + 2 delta) A + eps / 2 |exact|,     |lse - exact| <= delta + 2^-15 + 2^-22 |exact|."""
import math

import pytest
import torch

import block_sparse_attention_cov_b200 as sa
import ops_ref as ref
from block_sparse_attention_cov_b200 import _lib
from block_sparse_attention_cov_b200.build import build

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _blank(pages, heads, d):
    """A cache whose every byte is NaN, scales too: what no sequence holds must not matter."""
    c = sa.Cache.empty(pages, heads, d)
    c.k.view(torch.uint8).fill_(0x7F)
    c.v.view(torch.uint8).fill_(0xFF)
    c.k_scale.fill_(math.nan)
    c.v_scale.fill_(math.nan)
    return c


def _table(B, columns, pages, seed, unused=-1, lengths=None):
    """Scattered pages; columns behind a sequence's length hold `unused`."""
    t = torch.randperm(pages, generator=_gen(seed))[:B * columns].view(B, columns).to(torch.int32)
    if lengths is not None:
        for b, n in enumerate(lengths):
            t[b, (n + 63) // 64:] = unused
    return t


def _filled(lengths, heads, d, seed, spread=2.0, columns=None):
    """A cache holding `lengths` tokens of each sequence, rows behind them NaN, page scales spread over 2^+-spread."""
    B = len(lengths)
    columns = columns or max(1, (max(lengths) + 63) // 64)
    pages = B * columns + 2
    c = _blank(pages, heads, d)
    t = _table(B, columns, pages, seed, lengths=lengths)
    g = _gen(seed + 1)
    vals = []
    for name in ("k", "v"):
        x8 = getattr(c, name).cpu()
        xs = getattr(c, name + "_scale").cpu()
        for b, n in enumerate(lengths):
            for col in range((n + 63) // 64):
                rows = min(64, n - 64 * col)
                x = torch.randn((heads, rows, d), generator=g)
                x *= torch.exp2(spread * (2 * torch.rand((heads, 1, 1), generator=g) - 1))
                p = int(t[b, col])
                for h in range(heads):
                    s = ref.page_scale(x[h])
                    x8.view(torch.uint8)[p, h, :rows] = ref.to_e4m3(x[h], s).view(torch.uint8)
                    xs[p, h] = s
        getattr(c, name).view(torch.uint8).copy_(x8.view(torch.uint8))
        getattr(c, name + "_scale").copy_(xs)
        vals.append((x8, xs))
    return c, t, vals


def _values(vals, t, b, h, n):
    """fp64 [n, d] of what sequence b holds."""
    x8, xs = vals
    rows = [x8[int(t[b, col]), h].double() * float(xs[int(t[b, col]), h]) for col in range((n + 63) // 64)]
    return torch.cat(rows)[:n] if rows else torch.zeros((0, x8.shape[-1]), dtype=torch.float64)


def _check_attention(q, c, t, vals, lengths, counts, causal, out, lse, scale=None, skip=()):
    B, H, N, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out, lse, qc = out.cpu(), lse.cpu(), q.cpu()
    eps = torch.finfo(q.dtype).eps
    worst = 0.0
    for b in range(B):
        n = counts[b]
        for h in range(H):
            j = h // (H // c.heads)
            k, v = _values(vals[0], t, b, j, lengths[b]), _values(vals[1], t, b, j, lengths[b])
            o, l, mag, size = ref.attend(qc[b, h], k, v, causal, n, scale)
            delta = 2.0 ** -18 * size
            tol = (2.0 ** -11 + 2.0 ** -15 + 2 * delta)[:, None] * mag + eps / 2 * 1.01 * o.abs() + \
                torch.finfo(q.dtype).tiny * eps
            err = (out[b, h, :n].double() - o).abs()
            assert (err <= tol).all(), (b, h, float((err / tol.clamp(min=1e-30)).max()))
            empty = torch.isinf(l)
            assert torch.equal(torch.isinf(lse[b, h, :n]), empty)
            e2 = (lse[b, h, :n].double() - l)[~empty].abs()
            assert (e2 <= (delta + 2.0 ** -15 + 2.0 ** -22 * l.abs())[~empty]).all(), (b, h, float(e2.max()))
            worst = max(worst, float((err / tol.clamp(min=1e-30)).max()) if n else 0.0)
    return worst


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _attend(q, c, t, lengths, counts, causal, scale=None):
    """Through the public call, into marked outputs; checks that rows behind the queries keep their mark."""
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    ws = sa.cache_workspace(q, c, t)
    ws[_lib.WORKSPACE_BYTES:].fill_(0xFF)  # the rest of a workspace needs no initialisation
    sa.cache_attention(q, c, t.cuda(), _i32(lengths), counts=None if counts is None else _i32(counts), causal=causal,
                       scale=scale, out=out, lse=lse, ws=ws)
    assert sa.status(ws) == 0
    for b, n in enumerate(counts or []):
        assert (out[b, :, n:] == 7.0).all() and (lse[b, :, n:] == 7.0).all()
    return out, lse


ATTEND = [
    # H, Hk, N, d, lengths, counts, causal, dtype
    (1, 1, 1, 64, [1], None, True, torch.bfloat16),
    (4, 4, 1, 128, [63, 64, 65, 0], None, True, torch.bfloat16),
    (5, 1, 1, 128, [700], None, False, torch.float16),
    (8, 2, 1, 64, [129, 1, 2000], None, True, torch.bfloat16),
    (6, 2, 3, 128, [5, 130, 2], [3, 1, 3], True, torch.float16),        # 3 queries of a sequence of 2: a row sees nothing
    (12, 1, 4, 64, [333, 64], [4, 0], True, torch.bfloat16),            # 48 rows of one key head; a sequence without queries
    (17, 1, 1, 128, [450], None, False, torch.bfloat16),                # a group that is no tile
    (2, 2, 30, 128, [100, 20], [30, 20], True, torch.bfloat16),
    (2, 1, 65, 64, [65, 300], None, True, torch.float16),               # first shapes of the many-query kernel
    (3, 1, 100, 128, [257, 100], [100, 31], True, torch.bfloat16),
    (2, 2, 129, 128, [129], None, False, torch.bfloat16),
    (2, 2, 256, 64, [640, 0, 191], [256, 0, 191], True, torch.bfloat16),
    (5, 1, 333, 128, [1000], None, True, torch.float16),
    (1, 1, 600, 128, [600, 599], [600, 513], True, torch.bfloat16),
    (2, 1, 200, 64, [60], None, True, torch.bfloat16),                  # more queries than keys: 140 rows see nothing
    (1, 1, 300, 128, [64 * 70 + 3], None, False, torch.bfloat16),       # split key axis
]


@pytest.mark.parametrize("H,Hk,N,d,lengths,counts,causal,dtype", ATTEND)
def test_attention_against_formula(H, Hk, N, d, lengths, counts, causal, dtype):
    B = len(lengths)
    c, t, vals = _filled(lengths, Hk, d, seed=N + d)
    q = torch.randn((B, H, N, d), generator=_gen(9)).to(dtype).cuda()
    out, lse = _attend(q, c, t, lengths, counts, causal)
    print("worst share of the tolerance:", _check_attention(q, c, t, vals, lengths, counts or [N] * B, causal, out, lse))


@pytest.mark.parametrize("N", [1, 150])
def test_attention_long_table_short_sequences(N):
    """A table of many columns (so a split key axis) with sequences from none to many tokens."""
    lengths = [0, 1, 64, 200, 64 * 90 - 1]
    c, t, vals = _filled(lengths, 2, 128, seed=3, columns=90)
    counts = [min(N, n) for n in lengths]
    q = torch.randn((5, 4, N, 128), generator=_gen(10)).to(torch.bfloat16).cuda()
    for causal in (True, False):
        out, lse = _attend(q, c, t, lengths, counts, causal)
        _check_attention(q, c, t, vals, lengths, counts, causal, out, lse)


@pytest.mark.parametrize("B,Hk,N", [(33, 16, 1), (64, 8, 1), (65, 8, 1), (33, 16, 3)])
def test_attention_of_many_sequences(B, Hk, N):
    """More key heads than the GPU takes at once, sequences of equal, falling, rising and no length, with and without
    queries: each gets its own answer."""
    lengths = [(37 * b) % 150 if b % 5 else (0, 64, 150)[b % 3] for b in range(B)]
    counts = [min(n, N if b % 7 else 0) for b, n in enumerate(lengths)]
    c, t, vals = _filled(lengths, Hk, 64, seed=B + N)
    q = torch.randn((B, 2 * Hk, N, 64), generator=_gen(15)).to(torch.bfloat16).cuda()
    out, lse = _attend(q, c, t, lengths, counts, True)
    _check_attention(q, c, t, vals, lengths, counts, True, out, lse)


@pytest.mark.parametrize("N", [1, 90])
@pytest.mark.parametrize("size", [1e-30, 30.0, 1e4])
def test_attention_extreme_queries_and_scales(N, size):
    """Tiny queries (uniform weights), peaked ones, and huge ones (one key takes all); pages up to 2^24 apart."""
    lengths = [400]
    c, t, vals = _filled(lengths, 1, 64, seed=5, spread=12.0)
    q = (torch.randn((1, 2, N, 64), generator=_gen(11)) * size).to(torch.bfloat16).cuda()
    out, lse = _attend(q, c, t, lengths, None, False)
    _check_attention(q, c, t, vals, lengths, [N], False, out, lse)
    # another softmax scale
    out, lse = _attend(q, c, t, lengths, None, False, scale=0.01)
    _check_attention(q, c, t, vals, lengths, [N], False, out, lse, scale=0.01)


def test_attention_of_zero_queries_and_zero_values():
    c = sa.Cache.empty(3, 1, 64)
    c.k.view(torch.uint8).zero_(), c.v.view(torch.uint8).zero_()
    c.k_scale.fill_(2.0 ** -32), c.v_scale.fill_(2.0 ** -32)
    for N in (1, 100):
        q = torch.zeros((1, 1, N, 64), dtype=torch.bfloat16, device="cuda")
        out, lse = _attend(q, c, torch.tensor([[2, 0, 1]], dtype=torch.int32), [150], None, False)
        assert (out == 0).all()
        assert torch.allclose(lse, torch.full_like(lse, math.log(150)), atol=2.0 ** -15)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponent", [-32, 0, 6, 32])
def test_rows_that_see_nothing_at_any_value_scale(d, exponent):
    """200 queries of a sequence of 50 tokens: the first 150 rows give 0 and -inf, whatever the pages' scales; the others
    are finite."""
    c = sa.Cache.empty(1, 1, d)
    c.k.view(torch.uint8).random_(0, 0x70, generator=torch.Generator("cuda").manual_seed(1))
    c.v.view(torch.uint8).random_(0, 0x70, generator=torch.Generator("cuda").manual_seed(2))
    c.k_scale.fill_(0.01), c.v_scale.fill_(2.0 ** exponent)
    q = torch.randn((1, 2, 200, d), generator=_gen(14)).to(torch.bfloat16).cuda()
    out, lse = _attend(q, c, torch.zeros((1, 1), dtype=torch.int32), [50], None, True)
    assert (out[:, :, :150] == 0).all() and (lse[:, :, :150] == -math.inf).all()
    assert torch.isfinite(out).all() and torch.isfinite(lse[:, :, 150:]).all() and (out[:, :, 150:] != 0).any(-1).all()


@pytest.mark.parametrize("N", [3, 40, 150])
def test_attention_not_finite(N):
    """A NaN or infinite query makes its own row NaN; a NaN key or value reaches exactly the rows (and, for a value, the
    column) that see its token."""
    L = 64 * 5
    c, t, vals = _filled([L], 1, 128, seed=6)
    p, r = int(t[0, 4]), 62  # the sequence's last token but one: seen by the last two queries
    v0 = int(c.v.view(torch.uint8)[p, 0, r, 17])
    q = torch.randn((1, 2, N, 128), generator=_gen(12)).to(torch.bfloat16).cuda()
    clean, clean_lse = _attend(q, c, t, [L], None, True)
    c.v.view(torch.uint8)[p, 0, r, 17] = 0x7F
    out, lse = _attend(q, c, t, [L], None, True)
    nan = torch.isnan(out)
    assert nan[:, :, N - 2:, 17].all() and int(nan.sum()) == 2 * 2
    assert torch.equal(out[~nan], clean[~nan]) and torch.equal(lse, clean_lse)
    c.v.view(torch.uint8)[p, 0, r, 17] = v0
    c.k.view(torch.uint8)[p, 0, r, 5] = 0xFF
    out, lse = _attend(q, c, t, [L], None, True)
    nan = torch.isnan(out).all(-1)
    assert nan[:, :, N - 2:].all() and int(torch.isnan(out).sum()) == 2 * 2 * 128
    assert torch.isnan(lse[:, :, N - 2:]).all() and torch.equal(lse[:, :, :N - 2], clean_lse[:, :, :N - 2])
    assert torch.equal(out[:, :, :N - 2], clean[:, :, :N - 2])
    c.k.view(torch.uint8)[p, 0, r, 5] = 0
    clean, _ = _attend(q, c, t, [L], None, False)
    q[0, 1, 1, 3] = math.inf
    q[0, 0, 0, 9] = math.nan
    out, lse = _attend(q, c, t, [L], None, False)
    bad = torch.zeros((1, 2, N), dtype=torch.bool, device="cuda")
    bad[0, 1, 1] = bad[0, 0, 0] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("N", [2, 140])
def test_attention_strides_streams_and_repeats(N):
    lengths = [310, 77]
    c, t, vals = _filled(lengths, 2, 128, seed=7)
    B, H, d = 2, 6, 128
    q = torch.randn((B, H, N, d), generator=_gen(13)).to(torch.bfloat16).cuda()
    want, want_lse = _attend(q, c, t, lengths, None, True)
    # [B, N, H, d] order for queries and outputs, padded rows, a broadcast query
    qs = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    out = torch.empty((B, N, H, d + 8), dtype=q.dtype, device="cuda").permute(0, 2, 1, 3)[..., :d]
    sa.cache_attention(qs, c, t.cuda(), _i32(lengths), out=out)
    assert torch.equal(out, want)
    one = q[:, :1].expand(B, H, N, d)
    got, _ = sa.cache_attention(one, c, t.cuda(), _i32(lengths), out=torch.empty_like(q))
    assert torch.equal(got[:, 0], want[:, 0])  # the other heads share the query and, within the group, the keys
    assert torch.equal(got[:, 1], want[:, 0]) and torch.equal(got[:, 2], want[:, 0])
    # pages of one layer of a cache of three, a table cut from a wider one
    k3 = torch.zeros((c.pages, 3, c.heads, 64, d), dtype=torch.uint8, device="cuda").view(E4M3)
    v3, s3 = torch.zeros_like(k3.view(torch.uint8)).view(E4M3), torch.zeros((2, c.pages, 3, c.heads), device="cuda")
    k3.view(torch.uint8)[:, 1] = c.k.view(torch.uint8)
    v3.view(torch.uint8)[:, 1] = c.v.view(torch.uint8)
    s3[0, :, 1], s3[1, :, 1] = c.k_scale, c.v_scale
    layer = sa.Cache(k3[:, 1], v3[:, 1], s3[0, :, 1], s3[1, :, 1])
    wide = torch.full((B, t.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + t.shape[1]] = t.cuda()
    got, got_lse = sa.cache_attention(q, layer, wide[:, 2:2 + t.shape[1]], _i32(lengths))
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    # the same bits again, and from another stream than the tensors'
    ws = sa.cache_workspace(q, c, t)
    args = (q, c, t.cuda(), _i32(lengths))
    for _ in range(3):
        got, got_lse = sa.cache_attention(*args, ws=ws)
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = sa.cache_attention(*args, want_lse=False)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


APPEND = [
    # H, N, d, starts, counts, dtype
    (1, 1, 64, [0], None, torch.bfloat16),
    (3, 1, 128, [0, 63, 64, 65], None, torch.bfloat16),
    (2, 64, 128, [0, 1], None, torch.float16),
    (2, 65, 64, [10, 127], [65, 2], torch.float32),
    (4, 200, 128, [0, 30, 64], [200, 0, 131], torch.bfloat16),
    (1, 1000, 64, [5], [999], torch.float16),
]


@pytest.mark.parametrize("H,N,d,starts,counts,dtype", APPEND)
@pytest.mark.parametrize("order", ["bhnd", "bnhd"])
def test_append_bitwise(H, N, d, starts, counts, dtype, order):
    B = len(starts)
    n = counts or [N] * B
    columns = max((s + N + 63) // 64 for s in starts)
    c, t, _ = _filled(starts, H, d, seed=20, columns=columns, spread=3.0)
    full = _table(B, columns, c.pages, 20)  # the same permutation, every column named
    t = torch.where(t < 0, full, t)
    g = _gen(21)
    x = [torch.randn((B, H, N, d), generator=g) * torch.exp2(4 * torch.rand((B, H, N, 1), generator=g)) for _ in range(2)]
    x[0][:, :, 0, 0] = 448.0 if N > 1 else x[0][:, :, 0, 0]   # exactly at the border of a scale
    x = [y.to(dtype) for y in x]
    want = [(getattr(c, nm).cpu(), getattr(c, nm + "_scale").cpu()) for nm in ("k", "v")]
    for (x8, xs), y in zip(want, x):
        for b in range(B):
            ref.append(x8, xs, y[b], t[b], starts[b], n[b])
    dev = [y.cuda() if order == "bhnd" else y.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).cuda() for y in x]
    ws = sa.workspace()
    ws.zero_()
    lengths = _i32(starts)
    sa.cache_append(c, dev[0], dev[1], t.cuda(), lengths, counts=None if counts is None else _i32(counts), ws=ws)
    assert sa.status(ws) == 0 and lengths.tolist() == starts
    for (x8, xs), nm in zip(want, ("k", "v")):
        got8, got_s = getattr(c, nm).cpu().view(torch.uint8), getattr(c, nm + "_scale").cpu()
        assert torch.equal(got_s.view(torch.int32), xs.view(torch.int32))
        diff = got8 != x8.view(torch.uint8)
        # NaN may carry either sign
        both = torch.isnan(getattr(c, nm).cpu().float()) & torch.isnan(x8.float())
        assert not (diff & ~both).any()


def test_append_extremes():
    """Zeros, values beyond the largest scale, below the smallest, denormal, not finite; a page whose scale rises by
    2^40 under older tokens."""
    c = _blank(2, 1, 64)
    t = torch.tensor([[1, 0]], dtype=torch.int32)
    rows = torch.zeros((1, 1, 5, 64))
    rows[0, 0, 1, :4] = torch.tensor([2.0 ** -40, -(2.0 ** -44), 2.0 ** -30, 1e-42])
    rows[0, 0, 3, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    rows[0, 0, 4, :3] = torch.tensor([3.5, 1e30, -1e13])
    at = 0
    want = [(getattr(c, nm).cpu(), getattr(c, nm + "_scale").cpu()) for nm in ("k", "v")]
    for piece in ([0], [1], [3], [4], [2, 1]):
        x = rows[:, :, piece]
        sa.cache_append(c, x.cuda(), x.cuda(), t.cuda(), _i32([at]))
        for x8, xs in want:
            ref.append(x8, xs, x[0], t[0], at, len(piece))
        at += len(piece)
        for (x8, xs), nm in zip(want, ("k", "v")):
            assert torch.equal(getattr(c, nm + "_scale").cpu()[1], xs[1])
            a, b = getattr(c, nm).cpu()[1, 0, :at].float(), x8[1, 0, :at].float()
            assert torch.equal(a.nan_to_num(999.0), b.nan_to_num(999.0))
    assert float(c.k_scale[1, 0]) == 2.0 ** 32


@pytest.mark.parametrize("N", [1, 80])
@pytest.mark.parametrize("d", [64, 128])
def test_every_e4m3_value_is_read_exactly(N, d):
    """One key of every e4m3 value, subnormals and both signs, among otherwise zero keys: the outputs of queries that pick
    single dimensions are those values' softmax, and values come back as they are where one key takes all."""
    codes = torch.tensor([b for b in range(256) if b & 0x7F != 0x7F], dtype=torch.uint8)
    n = codes.numel()  # 254 tokens
    c = sa.Cache.empty(4, 1, d)
    c.k.view(torch.uint8).zero_(), c.v.view(torch.uint8).zero_()
    c.k_scale.fill_(1.0), c.v_scale.fill_(2.0 ** 5)
    flat_k, flat_v = c.k.view(torch.uint8).view(256, d), c.v.view(torch.uint8).view(256, d)
    for j in range(d):  # dimension j of token u holds code (u + 7 j)
        flat_v[:n, j] = codes.roll(-7 * j).cuda()
    marks = torch.randperm(n, generator=_gen(70))[:N]
    t = torch.arange(4, dtype=torch.int32).view(1, 4)
    for i, u in enumerate(marks.tolist()):  # key u alone has 448 in dimension i % d, and wins by far
        if i < d:
            flat_k[u, i] = 0x7E
    rows = min(N, d)
    q = torch.zeros((1, 1, N, d), dtype=torch.bfloat16)
    for i in range(rows):
        q[0, 0, i, i] = 8.0
    out, lse = sa.cache_attention(q.cuda(), c, t.cuda(), _i32([n]), causal=False)
    for i, u in enumerate(marks.tolist()[:rows]):
        want = flat_v[u].view(E4M3).double().cpu() * 32
        # the other 253 keys weigh e^-(448 * 8 / sqrt(d)) each: nothing
        assert torch.equal(out[0, 0, i].double().cpu(), want.to(torch.bfloat16).double())
    # keys: scores of every code through lse of two keys, the code's and a zero
    for code in (0x01, 0x07, 0x08, 0x81, 0x3C, 0x7E, 0xFE):
        flat_k.zero_()
        flat_k[0, 5] = code
        q = torch.zeros((1, 1, N, d), dtype=torch.bfloat16)
        q[..., 5] = 1.0
        value = float(torch.tensor([code], dtype=torch.uint8).view(E4M3).float())
        scale = 4.0 if abs(value) < 1 else 0.01
        _, lse = sa.cache_attention(q.cuda(), c, t.cuda(), _i32([1]), causal=False, scale=scale)
        assert torch.allclose(lse.cpu(), torch.full_like(lse.cpu(), value * scale), rtol=2.0 ** -20, atol=2.0 ** -20)


def test_token_by_token_equals_a_chunk_where_scales_agree():
    """Appending one by one ends with the scale of the whole page, and with its bytes save values that sank."""
    d, n = 128, 64
    x = torch.randn((1, 2, n, d), generator=_gen(30)).to(torch.bfloat16).cuda()
    a, b = sa.Cache.empty(1, 2, d), sa.Cache.empty(1, 2, d)
    t = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    sa.cache_append(a, x, x, t, _i32([0]))
    for i in range(n):
        sa.cache_append(b, x[:, :, i:i + 1], x[:, :, i:i + 1], t, _i32([i]))
    assert torch.equal(a.k_scale, b.k_scale)
    va, vb = a.k.float(), b.k.float()
    # two roundings of a value below e4m3's normal range (2^-6): at most one subnormal step (2^-9) apart
    assert torch.equal(torch.where(va.abs() >= 2.0 ** -6, va, 0), torch.where(va.abs() >= 2.0 ** -6, vb, 0))
    assert (va - vb).abs().max() <= 2.0 ** -9


def test_bad_pages_lengths_and_counts_are_reported_and_touch_nothing():
    H, d = 2, 64
    c, t, vals = _filled([200, 130], H, d, seed=40, columns=4)
    t[0, 1] = c.pages + 5     # a page that is not there
    t[1, 3] = -3              # behind the sequence: never read
    before = [x.clone() for x in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    for N in (1, 90):
        q = torch.randn((2, H, N, d), generator=_gen(41)).to(torch.bfloat16).cuda()
        ws = sa.cache_workspace(q, c, t)
        out, lse = sa.cache_attention(q, c, t.cuda(), _i32([200, 130]), causal=False, ws=ws)
        assert sa.status(ws) == _lib.ERR_PAGE
        # sequence 0 without the bad page's 64 tokens; sequence 1 as ever
        for h in range(H):
            keep = [i for i in range(200) if i // 64 != 1]
            rows = []
            for x8, xs in vals:
                tt = t.clone()
                tt[0, 1] = 0
                rows.append(_values((x8, xs), tt, 0, h, 200)[keep])
            o, l, mag, size = ref.attend(q[0, h].cpu(), rows[0], rows[1], False, N, d ** -0.5)
            tol = (2.0 ** -11 + 2.0 ** -15 + 2.0 ** -17 * size)[:, None] * mag + 2.0 ** -8 * 1.01 * o.abs()
            assert ((out[0, h].cpu().double() - o).abs() <= tol).all()
        _check_attention(q[1:], c, t[1:], vals, [130], [N], False, out[1:], lse[1:])
        # lengths and counts beyond the table and the tensor: clamped
        ws = sa.cache_workspace(q, c, t)
        good = torch.randperm(c.pages)[:8].view(2, 4).to(torch.int32).cuda()
        a, _ = sa.cache_attention(q, c, good, _i32([1 << 30, -7]), counts=_i32([N + 9, 1]), ws=ws)
        assert sa.status(ws) == _lib.ERR_PAGE
        w2 = sa.cache_workspace(q, c, t)
        b, _ = sa.cache_attention(q, c, good, _i32([256, 0]), counts=_i32([N, 1]), ws=w2)
        assert sa.status(w2) == 0
        assert torch.equal(a[0].nan_to_num(5.0), b[0].nan_to_num(5.0)) and (a[1, :, 0] == 0).all()
    x = torch.ones((2, H, 3, d), dtype=torch.bfloat16, device="cuda")
    for lengths, counts in (([-1, 300], [3, 3]), ([70, 1 << 30], [3, 3]), ([70, 256], [0, -1])):
        ws = sa.workspace()
        ws.zero_()
        sa.cache_append(c, x, x, t.cuda(), _i32(lengths), counts=_i32(counts), ws=ws)
        assert sa.status(ws) == _lib.ERR_PAGE
        for a, b in zip((c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale), before):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_offsets_beyond_32_bits():
    """A cache of more than 4 GiB: pages at its end and at its start."""
    H, d = 8, 128
    pages = 70000  # 64 KB each: 4.6 GB for keys and as much for values
    c = sa.Cache.empty(pages, H, d)
    t = torch.tensor([[pages - 1, 0, 69990, 65537]], dtype=torch.int32)
    x = torch.randn((1, H, 250, d), generator=_gen(50)).to(torch.bfloat16)
    y = torch.randn((1, H, 250, d), generator=_gen(51)).to(torch.bfloat16)
    sa.cache_append(c, x.cuda(), y.cuda(), t.cuda(), _i32([0]))
    small = [int(p) for p in t[0]]
    vals = [(getattr(c, nm)[small].cpu(), getattr(c, nm + "_scale")[small].cpu()) for nm in ("k", "v")]
    local = torch.arange(4).view(1, 4)
    for N in (1, 100):
        q = torch.randn((1, H, N, d), generator=_gen(52)).to(torch.bfloat16).cuda()
        out, lse = _attend(q, c, t, [250], None, False)
        _check_attention(q, c, local, vals, [250], [N], False, out, lse)


def test_together_as_a_decoder_uses_them():
    """Prompt, then single tokens: rotary, append and attention in a captured graph that is replayed with its lengths
    on the device, against dense() on the values that the cache holds (prompt) and the formula (steps)."""
    B, H, Hk, d, P, steps = 2, 4, 2, 64, 150, 5
    rope = sa.Rotary(d, layout="half", scaling=("yarn", 4.0, 128))
    g = _gen(60)
    cols = 4
    c = _blank(B * cols, Hk, d)
    t = torch.randperm(B * cols, generator=g)[:B * cols].view(B, cols).to(torch.int32)
    td = t.cuda()
    q = torch.randn((B, H, P, d), generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn((B, Hk, P, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    pos = torch.arange(P, dtype=torch.int32, device="cuda")
    q1, k1 = sa.rotary(q, k, rope, pos)
    sa.cache_append(c, k1, v, td, _i32([0, 0]))
    out, lse = sa.cache_attention(q1, c, td, _i32([P, P]))
    vals = [(getattr(c, nm).cpu(), getattr(c, nm + "_scale").cpu()) for nm in ("k", "v")]
    _check_attention(q1, c, t, vals, [P, P], [P, P], True, out, lse)

    lengths = _i32([P, P])
    sq = torch.empty((B, H, 1, d), dtype=torch.bfloat16, device="cuda")
    sk, sv = (torch.empty((B, Hk, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    so, sl = torch.empty_like(sq), torch.empty((B, H, 1), device="cuda")
    ws = sa.cache_workspace(sq, c, td)

    def step():
        rq, rk = sa.rotary(sq, sk, rope, lengths.view(B, 1))
        sa.cache_append(c, rk, sv, td, lengths)
        lengths.add_(1)
        sa.cache_attention(rq, c, td, lengths, out=so, lse=sl, ws=ws)
        return rq

    for x in (sq, sk, sv):
        x.zero_()
    keep = [x.clone() for x in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq = step()
    for x, y in zip((c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale), keep):
        x.copy_(y)
    lengths.fill_(P)
    for i in range(steps):
        for x in (sq, sk, sv):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        n = P + i + 1
        assert lengths.tolist() == [n, n] and sa.status(ws) == 0
        vals = [(getattr(c, nm).cpu(), getattr(c, nm + "_scale").cpu()) for nm in ("k", "v")]
        _check_attention(rq, c, t, vals, [n, n], [1, 1], True, so, sl)
