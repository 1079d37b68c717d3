"""The operators around attention in plain 64-bit torch on the CPU (tests only)."""
import math

import torch

BLOCK = 64
E4M3 = torch.float8_e4m3fn


def rotate(x, pos, freq, axis, rot, layout, gain=1.0, inverse=False):
    """x [B, H, N, d]; pos [B, N, axes] whole numbers; freq [rot / 2] radians per position; fp64."""
    x = x.double().cpu()
    pos = pos.double().cpu()
    out = x.clone()
    for p in range(rot // 2):
        i, j = (p, p + rot // 2) if layout == "half" else (2 * p, 2 * p + 1)
        a = pos[:, :, int(axis[p])] * float(freq[p]) * (-1 if inverse else 1)
        c, s = (gain * torch.cos(a))[:, None], (gain * torch.sin(a))[:, None]
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., j] * c + x[..., i] * s
    return out


def frequencies(pairs, theta=10000.0, scaling=None):
    """(frequencies, axes, gain) of the pairs of each axis."""
    freq, axis = [], []
    for a, n in enumerate(pairs):
        for i in range(n):
            base = theta
            if scaling and scaling[0] == "ntk":
                base = theta * scaling[1] ** (2 * n / (2 * n - 2))
            f = base ** (-i / n)
            if scaling and scaling[0] == "linear":
                f /= scaling[1]
            if scaling and scaling[0] == "yarn":
                fast, slow = (scaling[3], scaling[4]) if len(scaling) > 3 else (32.0, 1.0)
                keep = min(1.0, max(0.0, (scaling[2] * f / (2 * math.pi) - slow) / (fast - slow)))
                f = f * keep + f / scaling[1] * (1 - keep)
            freq.append(f)
            axis.append(a)
    gain = 0.1 * math.log(scaling[1]) + 1 if scaling and scaling[0] == "yarn" else 1.0
    return freq, axis, gain


def page_scale(x):
    """The smallest power of two s in 2^-32 .. 2^32 with max |x| <= 448 s, over finite elements."""
    x = x.double()
    top = float(torch.where(torch.isfinite(x), x.abs(), 0.0).max())
    e = -32
    while e < 32 and top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def to_e4m3(x, s):
    """x / s rounded to e4m3 (saturating; not finite: NaN). s is a power of two, so the division is exact in fp32."""
    y = (x.float() / s).clamp(-448, 448)
    return torch.where(torch.isfinite(x.float()), y, math.nan).to(E4M3)


def append(k8, ks, x, table, start, count):
    """Writes x [H, count.., d] of one sequence; k8 [pages, H, 64, d] (CPU float8) and ks [pages, H] change in place."""
    H = x.shape[0]
    raw = k8.view(torch.uint8)
    if count == 0:
        return
    for col in range(start // BLOCK, (start + count + BLOCK - 1) // BLOCK):
        lo, hi = max(start, col * BLOCK), min(start + count, (col + 1) * BLOCK)
        p, f = int(table[col]), lo - col * BLOCK
        for h in range(H):
            new = x[h, lo - start:hi - start]
            s = page_scale(new)
            if f > 0:
                old = float(ks[p, h])
                s = max(s, old)
                raw[p, h, :f] = to_e4m3(k8[p, h, :f].float() * old, s).view(torch.uint8)
            raw[p, h, f:hi - col * BLOCK] = to_e4m3(new, s).view(torch.uint8)
            ks[p, h] = s


def attend(q, k, v, causal, count, scale):
    """One head: q [N, d], k, v [L, d], the count first rows of q standing for the last tokens; fp64.
    Returns out, lse, and per element what the bounds need: sum p |v| / sum p and max sum |q||k| scale."""
    q, k, v = q.double(), k.double(), v.double()
    L = k.shape[0]
    out = torch.zeros(count, q.shape[1], dtype=torch.float64)
    lse = torch.full((count,), -math.inf, dtype=torch.float64)
    mag = torch.zeros_like(out)
    size = torch.zeros(count, dtype=torch.float64)
    for i in range(count):
        n = max(0, min(L, L - count + i + 1)) if causal else L
        if n == 0:
            continue
        s = (k[:n] @ q[i]) * scale
        lse[i] = torch.logsumexp(s, 0)
        p = torch.exp(s - lse[i])
        out[i] = p @ v[:n]
        mag[i] = p @ v[:n].abs()
        size[i] = ((k[:n].abs() @ q[i].abs()) * scale).max()
    return out, lse, mag, size
