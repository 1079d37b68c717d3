"""The cache's calls as programs make them: waits that run out, two calls at once, captured and replayed with other
lengths, graphs that share a workspace, a video stream of frames through rotary positions, cache and attention."""
import math

import pytest
import torch

import block_sparse_attention_cov_b200 as sa
import ops_ref as ref
from block_sparse_attention_cov_b200 import _lib
from block_sparse_attention_cov_b200.build import build
from block_sparse_attention_cov_b200.inputs import grid_positions
from hooklib import hooks_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _problem(B, H, Hk, N, d, lengths, columns, seed):
    g = torch.Generator().manual_seed(seed)
    c = sa.Cache.empty(B * columns, Hk, d)
    t = torch.randperm(B * columns, generator=g).view(B, columns).to(torch.int32).cuda()
    n = max(lengths)
    k, v = (torch.randn((B, Hk, n, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    sa.cache_append(c, k, v, t, _i32([0] * B), counts=_i32(lengths))
    q = torch.randn((B, H, N, d), generator=g).to(torch.bfloat16).cuda()
    return q, c, t


@pytest.mark.parametrize("N,d", [(1, 128), (3, 64), (300, 128), (300, 64)])
def test_expired_wait_reports_timeout_and_next_call_succeeds(N, d, monkeypatch):
    """In the test-hook build the first parts' first page is never requested: their waits run out after 20 ms, the call
    ends and says so, and the next call on a cleared status gives the product library's bits."""
    q, c, t = _problem(2, 4, 2, N, d, [700, 333], 11, 1)
    lengths = _i32([700, 333])
    want, want_lse = sa.cache_attention(q, c, t, lengths)
    ws = sa.cache_workspace(q, c, t)
    H = hooks_lib()
    monkeypatch.setattr(_lib, "_lib", H)
    assert H.solattn_test_set_hook(0, 20_000_000) == 0
    try:
        sa.cache_attention(q, c, t, lengths, ws=ws)
        assert sa.status(ws) == _lib.ERR_TIMEOUT
        words = ws[:16].view(torch.int32).tolist()
        assert words[1] == _lib.ERR_TIMEOUT and words[2] >= 40  # the wait site
    finally:
        assert H.solattn_test_set_hook(-1, 2_000_000_000) == 0
    sa.cache_attention(q, c, t, lengths, ws=ws)
    assert sa.status(ws) == _lib.ERR_TIMEOUT  # kept until it is cleared
    ws[:_lib.WORKSPACE_BYTES].zero_()
    out, lse = sa.cache_attention(q, c, t, lengths, ws=ws)
    assert sa.status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_calls_at_once():
    """Steps and chunks on two streams, each with its own workspace, many times over: the bits of the calls alone."""
    a = _problem(3, 8, 2, 1, 128, [3000, 17, 900], 47, 2)
    b = _problem(1, 2, 1, 400, 64, [1500], 24, 3)
    la, lb = _i32([3000, 17, 900]), _i32([1500])
    want = [sa.cache_attention(*a, la), sa.cache_attention(*b, lb)]
    wsa, wsb = sa.cache_workspace(a[0], a[1], a[2]), sa.cache_workspace(b[0], b[1], b[2])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            got.append((0, sa.cache_attention(*a, la, ws=wsa)))
        with torch.cuda.stream(s2):
            got.append((1, sa.cache_attention(*b, lb, ws=wsb)))
    torch.cuda.synchronize()
    assert sa.status(wsa) == 0 and sa.status(wsb) == 0
    for i, (o, l) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


@pytest.mark.parametrize("N", [1, 200])
def test_graph_follows_lengths_table_and_contents(N):
    """One capture, replayed with other lengths, another table and other queries; and two graphs on one workspace,
    replayed in turn."""
    columns = 20
    q, c, t = _problem(2, 4, 2, N, 128, [1280, 1280], columns, 4)
    lengths, counts = _i32([1280, 600]), _i32([N, N // 2 + 1])
    out, lse = torch.empty_like(q), torch.empty((2, 4, N), device="cuda")
    out2, lse2 = torch.empty_like(q), torch.empty((2, 4, N), device="cuda")
    ws = sa.cache_workspace(q, c, t)
    sa.cache_attention(q, c, t, lengths, counts=counts, out=out, lse=lse, ws=ws)
    graphs = []
    for o, l, causal in ((out, lse, True), (out2, lse2, False)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sa.cache_attention(q, c, t, lengths, counts=counts, causal=causal, out=o, lse=l, ws=ws)
        graphs.append(g)
    for i, (la, ca) in enumerate((([1280, 600], [N, 1]), ([5, 0], [min(N, 5), 0]), ([64, 1279], [1, N]))):
        lengths.copy_(_i32(la)), counts.copy_(_i32(ca))
        t.copy_(t.flip(1))
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        for o in (out, lse, out2, lse2):
            o.fill_(3.0)
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        assert sa.status(ws) == 0
        for o, l, causal in ((out, lse, True), (out2, lse2, False)):
            w, wl = torch.full_like(q, 3.0), torch.full_like(lse, 3.0)
            sa.cache_attention(q, c, t, lengths, counts=counts, causal=causal, out=w, lse=wl)
            assert torch.equal(o, w) and torch.equal(l, wl)


def test_stream_of_frames():
    """A video read frame by frame: each frame's queries and keys turned by their (t, h, w), keys and values written
    behind the earlier frames', and the frame attending all of them, against plain 64-bit attention on unrounded keys.

    The cache holds keys and values to 2^-4 of themselves at most (e4m3's half step): scores move by up to
    2^-4 sum |q||k| scale, which a softmax of this size turns into a few percent of the output's size; the check is
    that the error's norm stays below 8 percent, which a wrong frame, position or page exceeds by far (checked: the
    frames' order reversed gives over 50 percent)."""
    frames, gh, gw, H, d = 4, 6, 10, 2, 64
    F = gh * gw
    pairs = (12, 10, 10)
    rope = sa.Rotary(d, layout="interleaved", sections=pairs)
    freq, axis, _ = ref.frequencies(pairs)
    pos = grid_positions((frames, gh, gw)).to(torch.int32)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((1, H, frames * F, d), generator=g).to(torch.bfloat16) for _ in range(3))
    columns = (frames * F + 63) // 64
    c = sa.Cache.empty(columns, H, d)
    t = torch.randperm(columns, generator=g).view(1, columns).to(torch.int32).cuda()
    lengths = _i32([0])
    tq, tk = (ref.rotate(x, pos[None], freq, axis, d, "interleaved") for x in (q, k))
    for f in range(frames):
        part = slice(f * F, (f + 1) * F)
        pf = pos[part].contiguous().cuda()
        qf, kf = sa.rotary(q[:, :, part].cuda(), k[:, :, part].cuda(), rope, pf)
        sa.cache_append(c, kf, v[:, :, part].cuda(), t, lengths)
        lengths += F
        out, _ = sa.cache_attention(qf, c, t, lengths, causal=False)
        for h in range(H):
            o, *_ = ref.attend(tq[0, h, part], tk[0, h, :(f + 1) * F], v[0, h, :(f + 1) * F].double(), False, F, d ** -0.5)
            assert (out[0, h].cpu().double() - o).norm() <= 0.08 * o.norm()
            if f == frames - 1:
                wrong = tk[0, h].view(frames, F, d).flip(0).reshape(-1, d)
                w, *_ = ref.attend(tq[0, h, part], wrong, v[0, h].double(), False, F, d ** -0.5)
                assert (w - o).norm() > 0.5 * o.norm()
