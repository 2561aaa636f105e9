"""Plain 64-bit forms of the operators on a cache held in 8 bits and of the
verification of drafted tokens, and draws, for their tests."""
from __future__ import annotations

import math

import torch

import cache_refs as ref

E4M3 = torch.float8_e4m3fn


def round_e4m3(x):
    """fp64 values to the nearest e4m3 values (ties to even), as fp64: steps of 2^-3 of the leading power, 2^-9 at
    least; infinities and NaN to NaN."""
    fine = torch.isfinite(x)
    y = torch.where(fine, x, torch.zeros_like(x))
    e = torch.frexp(y)[1]
    step = ((e - 4).clamp(min=-9).long() + 1023 << 52).view(torch.float64)  # (exact on every device)
    return torch.where(fine, (y / step).round() * step, torch.full_like(y, math.nan))


def least_scale(a):
    """The least power of two, 2^-100 or more, with a <= 448 times it (a Python float)."""
    s = 2.0 ** -100
    if a > 448.0 * s:
        s = 2.0 ** (math.frexp(a)[1] - 10)
        while a > 448.0 * s:
            s *= 2.0
    return s


def values(codes, scale, block):
    """fp64 values [B, Hkv, Nk, d] of a cache."""
    return codes.double() * scale.double().repeat_interleave(block, -1)[..., :codes.shape[2], None]


def cache(g, B, Hkv, Nk, d, block, layout="bhnd", spread=0):
    """Codes and scales of random rows; `spread`: scales differ by up to 2^spread from block to block."""
    shape = {"bhnd": (B, Hkv, Nk, d), "bnhd": (B, Nk, Hkv, d), "pitch": (B, Hkv, Nk, d + 48)}[layout]
    nb = -(-Nk // block)
    x = torch.randn(B, Hkv, Nk, d, generator=g, device="cuda") * 60.0
    codes = torch.zeros(shape, device="cuda").to(E4M3)
    codes = codes.transpose(1, 2) if layout == "bnhd" else codes[..., 16:16 + d] if layout == "pitch" else codes
    codes.copy_(x.clamp(-448, 448).to(E4M3))
    e = torch.randint(-spread, spread + 1, (B, Hkv, nb), generator=g, device="cuda")
    return codes, (e - 6 + 127 << 23).to(torch.int32).view(torch.float32)


def append(x, n, codes, scale, block):
    """One head: x [N, d] (fp64) become the last N of n rows of codes [Nk, d] and scale [blocks]; (values as codes,
    scales), both fp64."""
    codes, scale = codes.double().clone(), scale.double().clone()
    N, Nk = x.shape[0], codes.shape[0]
    start = n - N
    rows = range(max(0, start), min(n, Nk))
    for blk in sorted({r // block for r in rows}):
        new = [r for r in rows if r // block == blk]
        y = x[[r - start for r in new]]
        a = y[torch.isfinite(y)].abs()
        s = least_scale(float(a.max()) if a.numel() else 0.0)
        old = range(blk * block, max(blk * block, min(start, Nk)))
        if len(old):
            s = max(s, float(scale[blk]))
            codes[old] = round_e4m3(codes[old] * (float(scale[blk]) / s))
        codes[new] = round_e4m3(y / s)
        scale[blk] = s
    return codes, scale


def compact(src, scale, dst, scale_out, kept, base, block):
    """One head: dst and scale_out (fp64 copies) after the move; entries that are not defined are NaN."""
    Nk, Nout = src.shape[0], dst.shape[0]
    out, so = dst.clone(), scale_out.clone()
    moves = {base + i: base + f for i, f in enumerate(kept) if f >= 0 and 0 <= base + f < Nk and 0 <= base + i < Nout}
    for blk in sorted({r // block for r in moves}):
        rows = {r: (src[f], float(scale[f // block])) for r, f in moves.items() if r // block == blk}
        if blk == max(base, 0) // block:
            for r in range(blk * block, max(base, 0)):
                rows[r] = (dst[r], float(scale_out[blk]))
        s = max(x[1] for x in rows.values())
        out[blk * block:(blk + 1) * block] = math.nan
        for r, (x, old) in rows.items():
            out[r] = round_e4m3(x * (old / s))
        so[blk] = s
    return out, so


def attention(q, k, v, mask, scale):
    """ref.attention, with what bounds its rounding: (o, lse, sum_j P |v|, the greatest scale * sum |q k|)."""
    o, lse, _ = ref.attention(q, k, v, mask, scale)
    use = mask.any(0)
    if not bool(use.any()):
        return o, lse, torch.zeros_like(o), 0.0
    k, v, mask = k[use].double(), v[use].double(), mask[:, use].to(q.device)
    p = torch.where(mask, (q.double() @ k.T * scale - lse[:, None].clamp(min=-1e30)).exp(), torch.zeros((), device=q.device,
                                                                                                    dtype=torch.float64))
    return o, lse, p @ v.abs(), float((q.double().abs() @ k.abs().T).max()) * abs(scale)


def verify(parents, tokens, target, draft, uniforms):
    """One sequence, its children in order (Python numbers; sums exact): (accepted nodes, the next token)."""
    Nt, V = len(parents), len(target[0])
    if parents[0] != -1:
        return [], -1
    path = [0]
    while True:
        n = path[-1]
        R, S, hit = list(target[n]), 1.0, None
        for i in range(n + 1, Nt):
            x = tokens[i]
            if parents[i] != n or not 0 <= x < V:
                continue
            qx = 1.0 if draft is None else draft[n][x]
            if uniforms[i] * qx * S < R[x]:
                hit = i
                break
            if draft is None:
                R[x] = max(R[x] - S, 0.0)
            else:
                R = [max(r - S * q, 0.0) for r, q in zip(R, draft[n])]
            S = math.fsum(R)
        if hit is None:
            break
        path.append(hit)
    if not math.fsum(R) > 0.0:
        R = list(target[n])
    total, below = math.fsum(R), 0.0
    if total <= 0.0:
        return path, -1
    for y, r in enumerate(R):
        below += r
        if below > uniforms[0] * total:
            return path, y
    return path, max(y for y, r in enumerate(R) if r > 0.0)
