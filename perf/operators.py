"""What is measured of the operators around attention: rotary positions (alone and fused with the pooled statistics),
and a cache of keys and values held in 8 bits (writing tokens into it, attention over it).

`run` computes them in plain torch operations where `own` is false, and through the package's public calls where it is
true. Shapes are those of the package's own workloads (45 x 80 latent frames, 40 / 24 / 8 heads, d 64 and 128, up to
262,144 tokens) and generic ones.

Cache: pages of 64 tokens, e4m3 values [pages][heads][64][d] and one fp32 scale (a power of two) per page and head for
keys and one for values; value = e4m3 * scale. A table [B][columns] gives the page of each 64-token block.
"""
import math
import random

import torch

own = False

BLOCK = 64
FRAME_H, FRAME_W = 45, 80
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCALE_EXP = 32  # page scales are 2^-32 .. 2^32
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one new token of each of 64 sequences at far positions, shared key heads, context stretched 8 times
        dict(name="rotary_step", op="rotary", B=64, H=40, Hk=8, N=1, d=128, rot=128, layout="half", axes=1,
             scaling="yarn", dtype="bf16", order="bhnd", inverse=False, far=262143),
        # queries and keys of 21 latent frames with (t, h, w) positions, heads next to each other as a projection
        # leaves them
        dict(name="rotary_video", op="rotary", B=1, H=40, Hk=40, N=75600, d=128, rot=128, layout="interleaved", axes=3,
             scaling="none", dtype="bf16", order="bnhd", inverse=False, far=0),
        # part of the head, odd length, backwards (the gradient's direction)
        dict(name="rotary_part_back", op="rotary", B=3, H=12, Hk=4, N=1001, d=64, rot=32, layout="half", axes=1,
             scaling="linear", dtype="fp16", order="bhnd", inverse=True, far=9000),
        # what stands before the sparse forward: a small clip, and 32768 tokens of 24 heads
        dict(name="rotary_pool_clip", op="rotary_pool", B=1, H=2, N=2048, d=64, rot=64, layout="interleaved", axes=3),
        dict(name="rotary_pool_frames", op="rotary_pool", B=1, H=24, N=32768, d=128, rot=128, layout="half", axes=3),
        # one token of each of 64 sequences behind up to 4096 cached ones: latency
        dict(name="append_step", op="append", B=64, H=8, N=1, d=128, past=4096, dtype="bf16", ragged=True),
        # a chunk of odd length for a ragged batch whose pages are part full
        dict(name="append_chunk", op="append", B=5, H=8, N=777, d=64, past=1500, dtype="fp16", ragged=True),
        # the whole of a 75600-token clip
        dict(name="append_video", op="append", B=1, H=40, N=75600, d=128, past=0, dtype="bf16", ragged=False),
        # one token over a short cache: latency
        dict(name="attend_one", op="attend", B=1, H=8, Hk=8, N=1, d=128, past=777, causal=True, dtype="bf16",
             ragged=False),
        # one token of each of 32 sequences of up to 32K tokens, 5 query heads to a key head: bandwidth
        dict(name="attend_step", op="attend", B=32, H=40, Hk=8, N=1, d=128, past=32700, causal=True, dtype="bf16",
             ragged=True),
        # a ragged causal chunk, d = 64, 3 query heads to a key head
        dict(name="attend_chunk", op="attend", B=3, H=12, Hk=4, N=1111, d=64, past=2000, causal=True, dtype="fp16",
             ragged=True),
        # a new latent frame against 21 cached ones (itself among them)
        dict(name="attend_frame", op="attend", B=1, H=8, Hk=8, N=3600, d=128, past=72000, causal=False, dtype="bf16",
             ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "rotary_pool", "append", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    if op == "rotary":
        N = _log(rng, 1, 60000)
        Hk = rng.choice([1, 2, 4, 8, 24])
        H = Hk * rng.choice([1, 1, 3, 5])
        B = _log(rng, 1, max(1, min(64, 2_000_000 // (N * (H + Hk)))))
        axes = rng.choice([1, 1, 3])
        rot = d if axes == 3 else rng.choice([d, d, d // 2, d // 4, d - 16])
        return dict(op=op, B=B, H=H, Hk=Hk, N=N, d=d, rot=rot, layout=rng.choice(["half", "interleaved"]), axes=axes,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]) if axes == 1 else "none",
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), order=rng.choice(["bhnd", "bnhd"]),
                    inverse=rng.random() < 0.3, far=rng.choice([0, 5000, 200000]))
    if op == "rotary_pool":
        N = _log(rng, 1, 30000)
        H = _log(rng, 1, 24)
        return dict(op=op, B=rng.choice([1, 1, 2]), H=H, N=N, d=d, rot=d, layout=rng.choice(["half", "interleaved"]),
                    axes=rng.choice([1, 3]))
    if op == "append":
        N = _log(rng, 1, 30000)
        H = rng.choice([1, 4, 8, 24])
        B = _log(rng, 1, max(1, min(64, 300_000 // (N * H))))
        return dict(op=op, B=B, H=H, N=N, d=d, past=rng.choice([0, _log(rng, 1, 8000)]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), ragged=rng.random() < 0.6)
    Hk = rng.choice([1, 2, 4, 8])
    H = Hk * rng.choice([1, 2, 3, 5, 8])
    if rng.random() < 0.55:  # a step: one token or a few
        N = rng.choice([1, 1, 1, 2, 4, 7])
        past = _log(rng, 1, 40000)
        B = _log(rng, 1, max(1, min(48, 3_000_000 // (past * Hk))))
    else:  # a chunk
        N = _log(rng, 16, 2500)
        past = _log(rng, 1, 20000)
        B = _log(rng, 1, max(1, min(8, 400_000_000 // (N * H * (past + N)))))
    return dict(op=op, B=B, H=H, Hk=Hk, N=N, d=d, past=past, causal=rng.random() < 0.6,
                dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.6)


def _pasts(c):
    """Cached tokens of each sequence before the call."""
    if not c["ragged"]:
        return [c["past"]] * c["B"]
    r = random.Random(7)
    return [c["past"]] + [int(c["past"] * (0.25 + 0.75 * r.random())) for _ in range(c["B"] - 1)]


def _counts(c):
    """New tokens of each sequence."""
    if not c["ragged"]:
        return [c["N"]] * c["B"]
    r = random.Random(8)
    return [c["N"]] + [r.randint(max(1, c["N"] // 2), c["N"]) for _ in range(c["B"] - 1)]


def _pairs(c):
    """(query, key) pairs of one head."""
    n = 0
    for past, cnt in zip(_pasts(c), _counts(c)):
        n += cnt * past + cnt * (cnt + 1) // 2 if c["causal"] else cnt * (past + cnt)
    return n


def work(c):
    if c["op"] == "rotary":
        n = c["B"] * (c["H"] + c["Hk"]) * c["N"] * c["d"]
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * size + c["B"] * c["N"] * c["axes"] * 4, "flops": 3 * n}
    if c["op"] == "rotary_pool":
        n, nb = c["B"] * c["H"] * c["N"] * c["d"], (c["N"] + BLOCK - 1) // BLOCK
        blocks = c["B"] * c["H"] * nb * c["d"]
        stats = c["B"] * c["H"] * c["d"] * (c["d"] + 1) * 4
        return {"bytes": 5 * n * 2 + blocks * (3 * 4 + 2 * 2) + stats + c["B"] * c["N"] * c["axes"] * 4,
                "flops": 9 * n + 2 * blocks * c["d"]}
    if c["op"] == "append":
        n = sum(_counts(c)) * c["H"] * c["d"]
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * (size + 1), "flops": 4 * n}
    rows, d = sum(_counts(c)) * c["H"], c["d"]
    keys = sum(p + n for p, n in zip(_pasts(c), _counts(c))) * c["Hk"]
    return {"bytes": 2 * keys * d + 2 * keys // BLOCK * 4 + rows * (4 * d + 4), "flops": 4 * d * c["H"] * _pairs(c)}


# ---------------------------------------------------------------------------------------------------------------------
# rotary frequencies (radians per position) of every rotated pair, and the axis it turns with
# ---------------------------------------------------------------------------------------------------------------------
THETA, STRETCH, TRAINED = 10000.0, 8.0, 32768


def _sections(c):
    """Rotated pairs of each position axis."""
    pairs = c["rot"] // 2
    if c["axes"] == 1:
        return [pairs]
    side = pairs // 3
    return [pairs - 2 * side, side, side]


def _frequencies(c):
    freq, axis = [], []
    for a, n in enumerate(_sections(c)):
        theta = THETA
        if c.get("scaling") == "ntk":
            theta = THETA * STRETCH ** (2 * n / (2 * n - 2))
        for i in range(n):
            f = theta ** (-i / n)
            if c.get("scaling") == "linear":
                f /= STRETCH
            if c.get("scaling") == "yarn":
                turns = TRAINED * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
                f = f / STRETCH * (1 - keep) + f * keep
            freq.append(f)
            axis.append(a)
    gain = 0.1 * math.log(STRETCH) + 1.0 if c.get("scaling") == "yarn" else 1.0
    return freq, axis, gain


def _positions(c, dev, g):
    """int32 [B, N] (one axis) or [B, N, 3] ((t, h, w) of a raster of latent frames)."""
    n = torch.arange(c["N"], device=dev)
    if c["axes"] == 1:
        far = max(0, c.get("far", 0) - c["N"])
        start = torch.randint(0, far + 1, (c["B"], 1), device=dev, generator=g)
        return (start + n).to(torch.int32)
    frame = FRAME_H * FRAME_W
    start = torch.randint(0, 4, (c["B"], 1), device=dev, generator=g)
    t = start + n // frame
    h = (n % frame // FRAME_W).expand_as(t)
    w = (n % FRAME_W).expand_as(t)
    return torch.stack([t, h, w], -1).to(torch.int32).contiguous()


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _quantise(x):
    """e4m3 values and power-of-two scales of full pages x [pages, heads, 64, d]."""
    f, e = torch.frexp(x.abs().amax((2, 3)))
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(-SCALE_EXP, SCALE_EXP)
    s = torch.ldexp(torch.ones_like(f), e)
    return (x / s[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _cache(c, heads, totals, dev, g):
    """A cache with contents in scattered pages, and its table [B, columns]."""
    columns = (max(totals) + BLOCK - 1) // BLOCK
    need = c["B"] * columns
    pages = need + 3
    out = []
    for _ in range(2):
        q = torch.empty((pages + 1, heads, BLOCK, c["d"]), dtype=torch.float8_e4m3fn, device=dev)
        s = torch.empty((pages + 1, heads), dtype=torch.float32, device=dev)
        for at in range(0, pages + 1, 4096):  # in parts: the fp32 values of a large cache need not fit at once
            x = torch.randn((min(4096, pages + 1 - at), heads, BLOCK, c["d"]), device=dev, generator=g)
            x *= torch.exp2(1.5 * torch.randn((x.shape[0], heads, 1, 1), device=dev, generator=g).clamp(-2, 2))
            q[at:at + 4096], s[at:at + 4096] = _quantise(x)
        out += [q, s]
    table = torch.randperm(pages, device=dev, generator=g)[:need].view(c["B"], columns).to(torch.int32)
    return out, table


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed) * 1_000_003 + 17)
    s = {"case": c}

    def tensor(heads, n, dtype, order="bhnd"):
        shape = (c["B"], n, heads, c["d"]) if order == "bnhd" else (c["B"], heads, n, c["d"])
        x = torch.randn(shape, device=dev, generator=g, dtype=torch.float32).to(dtype)
        return x.permute(0, 2, 1, 3) if order == "bnhd" else x

    if c["op"] in ("rotary", "rotary_pool"):
        dtype = TYPES[c.get("dtype", "bf16")]
        order = c.get("order", "bhnd")
        s["q"], s["k"] = tensor(c["H"], c["N"], dtype, order), tensor(c.get("Hk", c["H"]), c["N"], dtype, order)
        if c["op"] == "rotary_pool":
            s["v"] = tensor(c["H"], c["N"], dtype)
        s["pos"] = _positions(c, dev, g)
        freq, axis, s["gain"] = _frequencies(c)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(axis, dtype=torch.int64, device=dev)
        if own:
            import block_sparse_attention_cov_b200 as sa
            kind = c.get("scaling", "none")
            scaling = None if kind == "none" else ("yarn", STRETCH, TRAINED) if kind == "yarn" else (kind, STRETCH)
            s["rope"] = sa.Rotary(c["rot"], layout=c["layout"], theta=THETA, sections=_sections(c), scaling=scaling)
        return s

    pasts, counts = _pasts(c), _counts(c)
    heads = c["H"] if c["op"] == "append" else c["Hk"]
    (s["ck"], s["ks"], s["cv"], s["vs"]), s["table"] = _cache(c, heads, [p + n for p, n in zip(pasts, counts)], dev, g)
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev)
    dtype = TYPES[c["dtype"]]
    if c["op"] == "append":
        s["lengths"] = torch.tensor(pasts, dtype=torch.int32, device=dev)
        s["k"], s["v"] = tensor(heads, c["N"], dtype, "bnhd"), tensor(heads, c["N"], dtype, "bnhd")
        s["k"] *= 2.0
    else:
        s["lengths"] = torch.tensor([p + n for p, n in zip(pasts, counts)], dtype=torch.int32, device=dev)
        s["q"] = tensor(c["H"], c["N"], dtype)
        # rows behind a sequence's queries stay as they are: they start as zeros on both sides
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["q"].shape[:3], dtype=torch.float32, device=dev)
    if own:
        import block_sparse_attention_cov_b200 as sa
        s["cache"] = sa.Cache(s["ck"][:-1], s["cv"][:-1], s["ks"][:-1], s["vs"][:-1])
        s["ws"] = sa.workspace() if c["op"] == "append" else sa.cache_workspace(s["q"], s["cache"], s["table"])
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _angles(c, s):
    """cos and sin [B, 1, N, pairs] in 32 bits of angles formed in 64."""
    pos = s["pos"].double()
    pos = pos[..., None] if c["axes"] == 1 else pos
    turn = pos[:, :, s["axis"]] * s["freq"]
    turn = (-turn if c.get("inverse") else turn)[:, None]
    return (turn.cos() * s["gain"]).float(), (turn.sin() * s["gain"]).float()


def _rotate(c, x, cos, sin):
    """x [B, H, N, d] rotated, in 32 bits."""
    x = x.float()
    r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["layout"] == "half":
        a, b = r.chunk(2, -1)
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _block_means(x):
    n = x.shape[2]
    nb = (n + BLOCK - 1) // BLOCK
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * BLOCK - n))
    valid = (n - BLOCK * torch.arange(nb, device=x.device)).clamp(max=BLOCK).float()
    return x.unflatten(2, (nb, BLOCK)).sum(3) / valid[:, None]


def _write(old8, old_s, x, table, lengths, counts):
    """Writes x [B, H, N, d] behind `lengths` tokens of each sequence; old8 and old_s, whose last page is spare, change."""
    B, H, N, d = x.shape
    W = (N + BLOCK - 1) // BLOCK + 1  # pages that the new tokens can touch
    dev = x.device
    start = lengths.long()[:, None]
    pos = start // BLOCK * BLOCK + torch.arange(W * BLOCK, device=dev)  # [B, W * 64]
    at = pos - start
    new = ((at >= 0) & (at < counts.long()[:, None])).view(B, W, BLOCK)
    touched = new.any(2)
    column = (start // BLOCK + torch.arange(W, device=dev)).clamp(max=table.shape[1] - 1)
    page = torch.where(touched, table.long().gather(1, column), old8.shape[0] - 1)  # [B, W]
    was = (pos < start).view(B, W, BLOCK)  # tokens that the page held before
    xs = x.float().gather(2, at.clamp(0, N - 1)[:, None, :, None].expand(B, H, W * BLOCK, d))
    xs = xs.view(B, H, W, BLOCK, d).transpose(1, 2)  # [B, W, H, 64, d]
    keep8, keep_s = old8.view(torch.uint8)[page], old_s[page]
    is_new, is_old = new[:, :, None, :, None], was[:, :, None, :, None]
    finite = torch.isfinite(xs)
    f, e = torch.frexp((xs.abs() * (finite & is_new)).nan_to_num(0.0, 0.0, 0.0).amax((3, 4)))
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(-SCALE_EXP, SCALE_EXP)
    scale = torch.ldexp(torch.ones_like(f), e)
    scale = torch.where(was.any(2)[:, :, None], torch.maximum(scale, keep_s), scale)
    values = torch.where(is_old, keep8.view(torch.float8_e4m3fn).float() * keep_s[..., None, None], xs)
    values = (values / scale[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX)
    values = torch.where(finite | is_old, values, math.nan).to(torch.float8_e4m3fn).view(torch.uint8)
    old8.view(torch.uint8)[page] = torch.where(is_new | is_old, values, keep8)
    old_s[page] = scale


def _attend(c, s):
    B, H, N, d = s["q"].shape
    Hk, G = c["Hk"], c["H"] // c["Hk"]
    L = s["table"].shape[1] * BLOCK
    page = s["table"].long()
    pos = torch.arange(L, device=page.device)
    length, count = s["lengths"].long()[:, None, None], s["counts"].long()[:, None, None]
    inside = pos < length  # [B, 1, L]
    k = (s["ck"][page].float() * s["ks"][page][..., None, None]).transpose(1, 2).reshape(B, Hk, L, d)
    v = (s["cv"][page].float() * s["vs"][page][..., None, None]).transpose(1, 2).reshape(B, Hk, L, d)
    v = torch.where(inside[..., None], v, 0.0)
    q = s["q"].float().view(B, Hk, G * N, d)
    row = torch.arange(N, device=page.device)[:, None]
    limit = length - count + row + 1 if c["causal"] else length + 0 * row
    seen = inside & (pos < limit)  # [B, N, L]
    seen = seen[:, None, None].expand(B, 1, G, N, L).reshape(B, 1, G * N, L)
    score = torch.where(seen, q @ k.transpose(2, 3) * d ** -0.5, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, p @ v / total, 0.0).view(B, H, N, d).to(s["q"].dtype)
    lse = (torch.log(total) + top).view(B, H, N)
    lse = torch.where(torch.isnan(lse), -math.inf, lse)
    there = (row < count)[:, None]  # [B, 1, N, 1]
    s["out"] = torch.where(there, out, s["out"])
    s["lse"] = torch.where(there[..., 0], lse, s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    c = s["case"]
    if own:
        return _run_own(c, s)
    if c["op"] == "rotary":
        cos, sin = _angles(c, s)
        return {"q": _rotate(c, s["q"], cos, sin).to(s["q"].dtype), "k": _rotate(c, s["k"], cos, sin).to(s["k"].dtype)}
    if c["op"] == "rotary_pool":
        cos, sin = _angles(c, s)
        q, k = _rotate(c, s["q"], cos, sin), _rotate(c, s["k"], cos, sin)
        kbar, vbar = _block_means(k), _block_means(s["v"])
        kmean = kbar.mean(2)
        dev = kbar - kmean[:, :, None]
        return {"q": q.to(s["q"].dtype), "k": k.to(s["k"].dtype), "qbar": _block_means(q), "kbar": kbar, "vbar": vbar,
                "kmean": kmean, "kcov": dev.transpose(2, 3) @ dev / kbar.shape[2]}
    if c["op"] == "append":
        _write(s["ck"], s["ks"], s["k"], s["table"], s["lengths"], s["counts"])
        _write(s["cv"], s["vs"], s["v"], s["table"], s["lengths"], s["counts"])
        return {"k": s["ck"][:-1], "v": s["cv"][:-1], "k_scale": s["ks"][:-1], "v_scale": s["vs"][:-1]}
    return _attend(c, s)


def _run_own(c, s):
    import block_sparse_attention_cov_b200 as sa
    if c["op"] == "rotary":
        q, k = sa.rotary(s["q"], s["k"], s["rope"], s["pos"], inverse=c["inverse"])
        return {"q": q, "k": k}
    if c["op"] == "rotary_pool":
        q, k, stats = sa.rotary_pool(s["q"], s["k"], s["v"], s["rope"], s["pos"])
        return {"q": q, "k": k, **{n: stats.view(n) for n in ("qbar", "kbar", "vbar", "kmean", "kcov")}}
    if c["op"] == "append":
        sa.cache_append(s["cache"], s["k"], s["v"], s["table"], s["lengths"], counts=s["counts"], ws=s["ws"])
        return {"k": s["ck"][:-1], "v": s["cv"][:-1], "k_scale": s["ks"][:-1], "v_scale": s["vs"][:-1]}
    out, lse = sa.cache_attention(s["q"], s["cache"], s["table"], s["lengths"], counts=s["counts"],
                                  causal=c["causal"], out=s["out"], lse=s["lse"], ws=s["ws"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the above
# ---------------------------------------------------------------------------------------------------------------------
def _turned(c, s, x):
    """Pairs as complex numbers times gain * e^(i angle), fp64."""
    pos = s["pos"].double().reshape(c["B"], c["N"], -1)
    out = x.double().clone()
    half = c["rot"] // 2
    for i in range(half):
        lo, hi = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        angle = pos[:, :, int(s["axis"][i])] * float(s["freq"][i]) * (-1.0 if c.get("inverse") else 1.0)
        z = torch.complex(x[..., lo].double(), x[..., hi].double())
        z = z * torch.polar(torch.full_like(angle, s["gain"]), angle)[:, None]
        out[..., lo], out[..., hi] = z.real, z.imag
    return out


def _exact_write(c, s, name8, name_s, x):
    got8, got_s = s[name8].double(), s[name_s].double()
    for b in range(c["B"]):
        start, count = int(s["lengths"][b]), int(s["counts"][b])
        for col in range(start // BLOCK, (start + count + BLOCK - 1) // BLOCK):
            lo, hi = max(start, col * BLOCK), min(start + count, (col + 1) * BLOCK)
            page = int(s["table"][b, col])
            rows = x[b, :, lo - start:hi - start].double()
            need = rows.abs().amax((1, 2)) / E4M3_MAX
            # a logarithm of 2^e may come out an ulp above e; the next value of any input type is 8e-8 above it
            bits = torch.ceil(torch.log2(need.clamp(min=2.0 ** -40)) - 1e-9)
            scale = torch.exp2(bits.clamp(-SCALE_EXP, SCALE_EXP))
            if lo > col * BLOCK:
                held = got_s[page].clone()
                scale = torch.maximum(scale, held)
                got8[page, :, :lo - col * BLOCK] *= (held / scale)[:, None, None]
            got8[page, :, lo - col * BLOCK:hi - col * BLOCK] = rows / scale[:, None, None]
            got_s[page] = scale
    return got8[:-1], got_s[:-1]


def _exact_attend(c, s):
    B, H, N, d = s["q"].shape
    out = torch.zeros((B, H, N, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros((B, H, N), dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        L, n = int(s["lengths"][b]), int(s["counts"][b])
        page = s["table"][b, :(L + BLOCK - 1) // BLOCK].long()
        for h in range(H):
            j = h // (H // c["Hk"])
            k = (s["ck"][page, j].double() * s["ks"][page, j].double()[:, None, None]).reshape(-1, d)[:L]
            v = (s["cv"][page, j].double() * s["vs"][page, j].double()[:, None, None]).reshape(-1, d)[:L]
            score = s["q"][b, h, :n].double() @ k.T / math.sqrt(d)
            if c["causal"]:
                score = score.masked_fill(torch.ones_like(score).triu(L - n + 1) > 0, -math.inf)
            lse[b, h, :n] = torch.logsumexp(score, -1)
            out[b, h, :n] = torch.softmax(score, -1) @ v
    return {"out": out, "lse": lse}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rotary":
        return {"q": _turned(c, s, s["q"]), "k": _turned(c, s, s["k"])}
    if c["op"] == "rotary_pool":
        q, k, v = _turned(c, s, s["q"]), _turned(c, s, s["k"]), s["v"].double()
        got = {"q": q, "k": k}
        for name, x in (("qbar", q), ("kbar", k), ("vbar", v)):
            got[name] = torch.stack([part.mean(2) for part in x.split(BLOCK, 2)], 2)
        got["kmean"] = got["kbar"].mean(2)
        got["kcov"] = (got["kbar"].transpose(2, 3) @ got["kbar"] / got["kbar"].shape[2]
                       - got["kmean"][..., :, None] * got["kmean"][..., None, :])
        return got
    if c["op"] == "append":
        k8, ks = _exact_write(c, s, "ck", "ks", s["k"])
        v8, vs = _exact_write(c, s, "cv", "vs", s["v"])
        return {"k": k8, "v": v8, "k_scale": ks, "v_scale": vs}
    return _exact_attend(c, s)
