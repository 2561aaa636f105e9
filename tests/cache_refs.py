"""Plain 64-bit forms of the cache operators, and draws, for their tests."""
from __future__ import annotations

import math

import torch

INF = math.inf


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def draw(g, B, H, N, d, layout="bhnd", mult=1.0):
    """bf16 N(0,1) * mult as a [B, H, N, d] view: stored so, as [B, N, H, d], or with padded rows."""
    if layout == "bnhd":
        return (torch.randn(B, N, H, d, generator=g, device="cuda") * mult).to(torch.bfloat16).transpose(1, 2)
    if layout == "pitch":
        return (torch.randn(B, H, N, d + 24, generator=g, device="cuda") * mult).to(torch.bfloat16)[..., 8:8 + d]
    return (torch.randn(B, H, N, d, generator=g, device="cuda") * mult).to(torch.bfloat16)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def rope(x, pos, freq, rot, interleaved, factor, sign=1.0):
    """x [B, H, N, d], pos [B, N] -> (fp64 result, per-element |x1| + |x2| of its pair)."""
    x = x.double()
    a = pos.double()[:, None, :, None] * freq.double() * sign
    c, s = a.cos() * factor, a.sin() * factor
    y, mag = x.clone(), torch.zeros_like(x)
    i1, i2 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    mag[..., i1] = mag[..., i2] = x1.abs() + x2.abs()
    return y, mag


def tree_mask(parents, n, Nt, Nk):
    """[Nt, Nk] bool of one sequence of n rows, by walking each node's ancestors."""
    n = max(0, min(n, Nk))
    base = n - Nt
    mask = torch.zeros(Nt, Nk, dtype=torch.bool)
    for i in range(Nt):
        path, x, live = [], i, True
        while live and x >= 0:
            path.append(x)
            up = parents[x]
            live = base + x >= 0 and -1 <= up < x
            x = up
        if live:
            mask[i, :max(0, base)] = True
            mask[i, [base + x for x in path]] = True
    return mask


def attention(q, k, v, mask, scale):
    """fp64 o, lse, and the spread sum_j P |v - o| of one head; k, v rows outside every mask are not read."""
    use = mask.any(0)
    q, k, v, mask = q.double(), k[use].double(), v[use].double(), mask[:, use].to(q.device)
    t = (q @ k.T * scale).masked_fill(~mask, -INF)
    lse = torch.logsumexp(t, -1) if t.shape[1] else torch.full((q.shape[0],), -INF, device=q.device,
                                                                dtype=torch.float64)
    p = torch.where(mask, (t - lse[:, None].clamp(min=-1e30)).exp(), torch.zeros_like(t))
    o = p @ v
    spread = torch.stack([(p[i][:, None] * (v - o[i]).abs()).sum(0) for i in range(q.shape[0])])
    return o, lse, spread


def key_weights(q, k, lse, n, causal, scale):
    """fp64 column sums of one cache head: q [G, Nq, d], k [Nk, d], lse [G, Nq]; rows past n are 0."""
    Nq, Nk = q.shape[1], k.shape[0]
    n = max(0, min(n, Nk))
    w = torch.zeros(Nk, dtype=torch.float64, device=q.device)
    if n == 0:
        return w
    on = torch.isfinite(lse)
    qq = torch.where(on[..., None], q.double(), torch.zeros((), dtype=torch.float64, device=q.device))
    t = qq @ k[:n].double().T * scale
    p = torch.where(on[..., None], (t - torch.where(on, lse, torch.zeros_like(lse)).double()[..., None]).exp(),
                    torch.zeros_like(t))
    if causal:
        see = torch.arange(n, device=q.device) <= n - Nq + torch.arange(Nq, device=q.device)[:, None]
        p = torch.where(see, p, torch.zeros_like(p))
    w[:n] = p.sum((0, 1))
    return w


def select(w, n, keep, first, recent):
    """Kept rows of one head (a list), by a sort of (weight, row) pairs; NaN below every number."""
    w = w.tolist()
    n = max(0, min(n, len(w)))
    if n <= keep:
        return list(range(n)) + [-1] * (keep - n)
    middle = sorted(range(first, n - recent), key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0.0, j))
    return (list(range(first)) + sorted(middle[:keep - first - recent]) + list(range(n - recent, n)))
