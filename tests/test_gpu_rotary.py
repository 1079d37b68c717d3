"""Rotary positions (solattn_rotary) and rotary positions with the pooled statistics (solattn_rotary_pool) against
plain 64-bit formulas.

Tolerance of one element y = gain (x0 cos - x1 sin): the rounding to its type, eps / 2 |y|, and the fp32 arithmetic.
The angle's fraction of a turn is a 24-bit float of up to half a turn (pi 2^-24 = 1.9e-7 rad), sine and cosine are good
to 2 ulp (1.2e-7), and the products and their difference round three times (1.8e-7): under 5e-7 gain (|x0| + |x1|);
1e-6 is allowed."""
import math

import pytest
import torch

import block_sparse_attention_cov_b200 as sa
import ops_ref as ref
from block_sparse_attention_cov_b200.build import build
from block_sparse_attention_cov_b200.inputs import grid_positions

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build()


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _pair_sum(x, rot, layout):
    """|x0| + |x1| at both elements of every pair, 0 behind the rotated part."""
    a = x.double().cpu().abs()
    out = torch.zeros_like(a)
    i = torch.arange(rot // 2)
    lo, hi = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    s = a[..., lo] + a[..., hi]
    out[..., lo], out[..., hi] = s, s
    return out


def _check(got, x, want, rot, layout, gain):
    fi = torch.finfo(got.dtype)
    tol = fi.eps / 2 * want.abs() * 1.01 + 1e-6 * gain * _pair_sum(x, rot, layout) + fi.tiny * fi.eps
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err - tol).max())


CASES = [
    # B, H, Hk, N, d, rot, layout, dtype, scaling, far
    (2, 3, 1, 1, 128, 128, "half", torch.bfloat16, None, 262143),
    (1, 8, 8, 65, 64, 64, "interleaved", torch.bfloat16, None, 0),
    (3, 5, 2, 130, 128, 64, "half", torch.float16, ("linear", 4.0), 1000),
    (1, 2, 1, 7, 64, 48, "half", torch.float32, ("ntk", 8.0), 2_000_000_000),
    (2, 1, 1, 33, 128, 112, "half", torch.bfloat16, ("yarn", 8.0, 4096), 100000),
    (1, 4, 4, 19, 80, 20, "interleaved", torch.float16, None, 50),      # scalar path: 20 is no whole chunk
    (1, 3, 1, 11, 6, 6, "half", torch.float32, None, 5),
    (1, 40, 8, 257, 128, 128, "interleaved", torch.bfloat16, ("yarn", 2.0, 8192, 16.0, 2.0), 8000),
    (64, 7, 1, 1, 64, 2, "interleaved", torch.bfloat16, None, 77),
]


@pytest.mark.parametrize("B,H,Hk,N,d,rot,layout,dtype,scaling,far", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_against_formula(B, H, Hk, N, d, rot, layout, dtype, scaling, far, inverse):
    freq, axis, gain = ref.frequencies([rot // 2], 10000.0, scaling)
    rope = sa.Rotary(rot, layout=layout, scaling=scaling)
    assert rope.gain == pytest.approx(gain, rel=1e-7)
    pos = (torch.arange(B * N).view(B, N) * 3 + far - 3 * B * N).to(torch.int32) if far else \
        torch.arange(B * N).view(B, N).to(torch.int32)  # negative ones too, where far is small
    q, k = _rand((B, H, N, d), dtype, 1), _rand((B, Hk, N, d), dtype, 2)
    q0, k0 = q.clone(), k.clone()
    q2, k2 = sa.rotary(q, k, rope, pos.cuda(), inverse=inverse)
    torch.cuda.synchronize()
    assert torch.equal(q, q0) and torch.equal(k, k0)
    for x, y in ((q, q2), (k, k2)):
        want = ref.rotate(x, pos[..., None], freq, axis, rot, layout, rope.gain, inverse)
        _check(y, x, want, rot, layout, rope.gain)
    alone, none = sa.rotary(q, None, rope, pos.cuda(), inverse=inverse)
    assert none is None and torch.equal(alone, q2)
    sa.rotary(q, k, rope, pos.cuda(), inverse=inverse, out=(q, k))  # in place
    assert torch.equal(q, q2) and torch.equal(k, k2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_strides_and_alignment(layout):
    """[B, N, H, d] order, padded rows, rows off 16-byte boundaries, a broadcast input: the contiguous result's bits."""
    B, H, N, d = 2, 6, 37, 64
    rope = sa.Rotary(d, layout=layout)
    pos = (torch.arange(N) * 11).to(torch.int32).cuda()
    x = _rand((B, H, N, d), torch.bfloat16, 3)
    want, _ = sa.rotary(x, None, rope, pos)
    bnhd = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    padded = torch.zeros((B, H, N, d + 8), dtype=x.dtype, device="cuda")[..., :d].copy_(x)
    odd = torch.zeros((B, H, N, d + 3), dtype=x.dtype, device="cuda")[..., 1:d + 1].copy_(x)
    for view in (bnhd, padded, odd):
        got, _ = sa.rotary(view, None, rope, pos)
        assert torch.equal(got, want)
        into = torch.full_like(odd, 9.0)
        sa.rotary(view, None, rope, pos, out=(into, None))
        assert torch.equal(into, want)
    one = x[:, :1].expand(B, H, N, d)
    got, _ = sa.rotary(one, None, rope, pos, out=(torch.empty_like(x), None))
    assert torch.equal(got, want[:, :1].expand(B, H, N, d))
    # positions of a batch: shared, per sequence, and as a column of a wider tensor
    wide = torch.zeros((B, N, 3), dtype=torch.int32, device="cuda")
    wide[..., 1] = pos
    got, _ = sa.rotary(x, None, rope, wide[..., 1])
    assert torch.equal(got, want)


@pytest.mark.parametrize("d,pairs", [(128, (22, 21, 21)), (64, (16, 8, 8))])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_axes_of_a_grid(d, pairs, layout):
    grid = (3, 5, 7)
    pos = grid_positions(grid).to(torch.int32)
    N = pos.shape[0]
    freq, axis, _ = ref.frequencies(pairs)
    rope = sa.Rotary(d, layout=layout, sections=pairs)
    q = _rand((1, 4, N, d), torch.bfloat16, 5)
    got, _ = sa.rotary(q, None, rope, pos.cuda())
    _check(got, q, ref.rotate(q, pos[None], freq, axis, d, layout), d, layout, 1.0)


def test_rotary_own_frequencies_and_nan_stay_in_place():
    d = 64
    freq = [0.5 / (1 + i) for i in range(d // 2 - 1)] + [-7.25]  # a negative one, and more than a turn per position
    rope = sa.Rotary(d, layout="half", frequencies=freq, gain=0.75)
    pos = torch.tensor([0, 1, -5, 12345], dtype=torch.int32)
    q = _rand((1, 2, 4, d), torch.float32, 6)
    got, _ = sa.rotary(q, None, rope, pos.cuda())
    _check(got, q, ref.rotate(q, pos[None, :, None], freq, [0] * (d // 2), d, "half", 0.75), d, "half", 0.75)
    part = sa.Rotary(32, layout="half")
    q[0, 0, 1, 40] = math.nan      # behind the rotated part
    q[0, 1, 2, 3] = math.inf       # in pair 3
    got, _ = sa.rotary(q, None, part, pos.cuda())
    bad = ~torch.isfinite(got)
    assert set(map(tuple, bad.nonzero().tolist())) == {(0, 0, 1, 40), (0, 1, 2, 3), (0, 1, 2, 19)}


def test_inverse_is_the_gradient():
    """Against autograd of the formula in 64 bits, against differences, and as the transpose: <R x, y> = <x, R' y>."""
    d, N = 64, 21
    scaling = ("yarn", 8.0, 64)
    freq, axis, _ = ref.frequencies([16], 10000.0, scaling)
    rope = sa.Rotary(32, layout="interleaved", scaling=scaling)
    pos = (torch.arange(N) * 5).to(torch.int32)
    x, dy = _rand((2, 3, N, d), torch.float32, 7), _rand((2, 3, N, d), torch.float32, 8)
    got, _ = sa.rotary(dy, None, rope, pos.cuda(), inverse=True)
    P = pos[None, :, None].expand(2, N, 1).double()
    leaf = x.double().cpu().requires_grad_()
    rows = []
    for p in range(16):
        a = P[:, :, 0] * freq[p]
        c, s = rope.gain * torch.cos(a)[:, None], rope.gain * torch.sin(a)[:, None]
        x0, x1 = leaf[..., 2 * p], leaf[..., 2 * p + 1]
        rows += [x0 * c - x1 * s, x1 * c + x0 * s]
    y = torch.cat([torch.stack(rows, -1), leaf[..., 32:]], -1)
    y.backward(dy.double().cpu())
    tol = 1e-6 * rope.gain * _pair_sum(dy, 32, "interleaved") + 2.0 ** -23 * leaf.grad.abs()
    assert ((got.double().cpu() - leaf.grad).abs() <= tol).all()
    # differences: the map is linear, so one step of any size is exact up to rounding
    e = torch.zeros_like(x)
    e[1, 2, 9, 5] = 0.5
    y1, _ = sa.rotary(x + e, None, rope, pos.cuda())
    y0, _ = sa.rotary(x, None, rope, pos.cuda())
    slope = float(((y1 - y0).double() * dy.double()).sum() / 0.5)
    # two elements of y of size under 8, rounded to 2^-24 and off by 1e-6 of their pair, times dy / 0.5
    assert slope == pytest.approx(float(got[1, 2, 9, 5]), abs=2e-4)
    a = float((y0.double() * dy.double()).sum())
    b = float((x.double() * got.double()).sum())
    assert a == pytest.approx(b, abs=1e-6 * float(_pair_sum(x, 32, "interleaved").sum() + x.abs().sum()) * 4)


POOL = [
    # B, H, N, d, layout, axes
    (1, 2, 1, 64, "half", 1),
    (2, 3, 63, 128, "interleaved", 3),
    (1, 5, 64 * 9 + 17, 128, "half", 3),
    (2, 9, 64 * 4 + 1, 64, "interleaved", 1),
    (1, 1, 64 * 30, 64, "half", 3),
]


@pytest.mark.parametrize("B,H,N,d,layout,axes", POOL)
def test_rotary_pool_against_formula(B, H, N, d, layout, axes):
    """q', k' are rotary()'s bits; the means of 64 rotated values are off by the values' own 1e-6 (|x0| + |x1|) and an
    fp32 sum of 64 (64 2^-24 of the mean magnitude); mean and covariance of the pooled keys follow from kbar."""
    pairs = [d // 2] if axes == 1 else [d // 2 - 2 * (d // 6), d // 6, d // 6]
    freq, axis, _ = ref.frequencies(pairs)
    rope = sa.Rotary(d, layout=layout, sections=pairs)
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(-50, 5000, (B, N, axes), generator=g, dtype=torch.int32)
    dev_pos = (pos[..., 0].contiguous() if axes == 1 else pos).cuda()
    q, k, v = (_rand((B, H, N, d), torch.bfloat16, s) for s in (11, 12, 13))
    q2, k2, st = sa.rotary_pool(q, k, v, rope, dev_pos)
    want_q, want_k = sa.rotary(q, k, rope, dev_pos)
    assert torch.equal(q2, want_q) and torch.equal(k2, want_k)
    nb = (N + 63) // 64
    for name, x, turned in (("qbar", q, True), ("kbar", k, True), ("vbar", v, False)):
        y = ref.rotate(x, pos, freq, axis, d, layout) if turned else x.double().cpu()
        mean = torch.stack([y[:, :, 64 * j:64 * j + 64].mean(2) for j in range(nb)], 2)
        size = _pair_sum(x, d, layout)
        tol = torch.stack([size[:, :, 64 * j:64 * j + 64].mean(2) for j in range(nb)], 2) * (1e-6 + 64 * 2.0 ** -24)
        assert ((st.view(name).double().cpu() - mean).abs() <= tol).all(), name
        if name == "kbar":
            kb = mean
    for name in ("kbar", "vbar"):
        assert torch.equal(st.view(name + "16"), st.view(name).to(torch.bfloat16))
    # kmean and kcov exactly as pool() forms them from this kbar: against 64-bit sums of it
    own = st.view("kbar").double().cpu()
    km = own.mean(2)
    cov = (own - km[:, :, None]).transpose(2, 3) @ (own - km[:, :, None]) / nb
    assert torch.allclose(st.view("kmean").double().cpu(), km, rtol=1e-5, atol=1e-6)
    assert torch.allclose(st.view("kcov").double().cpu(), cov, rtol=1e-5, atol=1e-6)
    assert torch.allclose(own, kb, atol=1e-4)
    # in place, and into the other layout
    a, b = q.clone(), k.clone()
    sa.rotary_pool(a, b, v, rope, dev_pos, out=(a, b))
    assert torch.equal(a, q2) and torch.equal(b, k2)
    o = [torch.empty((B, N, H, d), dtype=q.dtype, device="cuda").permute(0, 2, 1, 3) for _ in range(2)]
    sa.rotary_pool(q, k, v, rope, dev_pos, out=tuple(o), stats=st)
    assert torch.equal(o[0], q2) and torch.equal(o[1], k2)


def test_rotary_pool_then_forward():
    """The step as it is used: the sparse forward on the fused result against the one on separate calls."""
    B, H, N, d = 1, 3, 64 * 20 + 5, 128
    rope = sa.Rotary(d, layout="interleaved", sections=(22, 21, 21))
    pos = grid_positions((3, 18, 24))[:N].to(torch.int32).cuda()
    q, k, v = (_rand((B, H, N, d), torch.bfloat16, s) for s in (21, 22, 23))
    q2, k2, st = sa.rotary_pool(q, k, v, rope, pos)
    ws = sa.workspace()
    out, lse, dens = sa.forward(q2, k2, v, st, beta=-math.inf, ws=ws)  # keeps every block: independent of the means
    assert sa.status(ws) == 0
    dense, dense_lse = sa.dense(q2, k2, v)
    assert torch.equal(out, dense) and torch.equal(lse, dense_lse)
    # beta = +inf skips every block: weights e^s of pooled scores s, values vbar (the same on both sides). The means
    # differ by the elements' rounding to bf16, 2^-9 of the block's mean magnitude at most, so a score by
    # delta = 2^-9 d^-1/2 sum_e (mq_e |kbar_e| + |qbar_e| mk_e + 2^-9 mq_e mk_e), and the weighted mean of vbar by
    # 2 delta max |vbar| (e^(2 delta) - 1 <= 2.5 delta here), plus one bf16 rounding on each side
    sep = sa.pool(q2, k2, v)
    a, la, _ = sa.forward(q2, k2, v, st, beta=math.inf)
    b, lb, _ = sa.forward(q2, k2, v, sep, beta=math.inf)
    nb = (N + 63) // 64
    mq, mk = (torch.stack([x[:, :, 64 * j:64 * j + 64].double().abs().mean(2) for j in range(nb)], 2) for x in (q2, k2))
    qb, kb = sep.view("qbar").double().abs(), sep.view("kbar").double().abs()
    step = 2.0 ** -9
    delta = float((mq @ kb.transpose(2, 3) + qb @ mk.transpose(2, 3) + step * mq @ mk.transpose(2, 3)).max()) * step / d ** 0.5
    assert delta < 0.1
    top = float(sep.view("vbar").abs().max())
    assert (a.float() - b.float()).abs().max() <= 2.5 * delta * top + 2 * 2.0 ** -9 * top
    assert (la - lb).abs().max() <= delta + 1e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(72, 64), (128, 16), (128, 96), (88, 32), (64, 6)])
def test_what_is_behind_the_rotated_part_keeps_its_bits(d, rot, layout, dtype):
    """Any bits behind the rotated part (NaN payloads, infinities) are copied; the part before takes none of them."""
    g = torch.Generator().manual_seed(31)
    as_int = torch.int32 if dtype == torch.float32 else torch.int16
    info = torch.iinfo(as_int)
    x = _rand((2, 3, 21, d), dtype, 32)
    x[..., rot:] = torch.randint(info.min, info.max + 1, (2, 3, 21, d - rot), generator=g,
                                 dtype=torch.int64).to(as_int).cuda().view(dtype)
    pos = torch.arange(21, dtype=torch.int32, device="cuda") * 97
    y, _ = sa.rotary(x, None, sa.Rotary(rot, layout=layout), pos)
    assert torch.equal(y[..., rot:].contiguous().view(as_int), x[..., rot:].contiguous().view(as_int))
    freq, axis, gain = ref.frequencies([rot // 2])
    _check(y[..., :rot], x[..., :rot], ref.rotate(x[..., :rot], pos.cpu()[None, :, None], freq, axis, rot, layout),
           rot, layout, 1.0)
