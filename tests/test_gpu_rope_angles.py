"""The angles of the rotary calls, against whole-number arithmetic.

The stated precision: within 2^-25 of a turn for every 32-bit position and
frequencies up to 128 radians per position.  A bf16 result shows an angle that
finely only where it nearly cancels, so each pair (x1, x2) is the one of 8-bit
mantissas whose y1 = x1 cos a - x2 sin a comes nearest to zero.

Bound of y1, relative to |x1| + |x2|: 2 pi 2^-25 < 2^-22.3 from the angle;
2^-22 from sine and cosine (two units in the last place, sincospif's bound);
2^-23 from two products and a difference in fp32; and half a bf16 step, 2^-8,
of y1 itself.
"""
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import fa_rope, fa_rope_append, fa_rope_frequencies

pytestmark = pytest.mark.gpu

BITS = 400


def _pi():
    """pi * 2^BITS, by pi = 16 atan(1/5) - 4 atan(1/239)."""
    def atan_inv(n):
        one = 1 << (BITS + 32)
        t = one // n
        s, k = t, 1
        while t:
            t //= n * n
            k += 2
            s += -(t // k) if k % 4 == 3 else t // k
        return s
    return (16 * atan_inv(5) - 4 * atan_inv(239)) >> 32


TWO_PI = 2 * _pi()


def angle(pos, f):
    """pos * f modulo a turn, in radians, in [-pi, pi): exact before the last rounding (f: a Python float)."""
    num, den = f.as_integer_ratio()
    a = pos * num * (1 << BITS) // den % TWO_PI
    if 2 * a >= TWO_PI:
        a -= TWO_PI
    return a / (1 << BITS)


def nearest_pair(a):
    """Mantissas and a power of two, (x1, x2), with x1 cos a - x2 sin a as near to zero as 8 bits allow."""
    c, s = math.cos(a), math.sin(a)
    if abs(s) < 2.0 ** -30 * abs(c):
        return 0.0, 1.0
    if abs(c) < 2.0 ** -30 * abs(s):
        return 1.0, 0.0
    t = s / c
    best = None
    e = math.frexp(abs(t))[1]          # |t| in [2^(e-1), 2^e)
    for k in (e, e - 1):
        for m2 in range(128, 256):
            m1 = round(abs(t) * 2.0 ** -k * m2)
            if 128 <= m1 <= 255:
                x1, x2 = math.copysign(m1 * 2.0 ** k, t), float(m2)
                err = abs(x1 * c - x2 * s) / (abs(x1) + x2)
                if best is None or err < best[0]:
                    best = (err, x1, x2)
    return best[1], best[2]


POSITIONS = [0, 1, -1, 7, 1000, 65535, 1 << 24, (1 << 24) + 1, 123456789, -987654321, 2 ** 31 - 1, -2 ** 31]


def tables():
    plain = fa_rope_frequencies(32, device="cpu")[0].tolist()
    parts = fa_rope_frequencies(32, scaling="by_parts", factor=16.0, device="cpu")[0].tolist()
    odd = torch.tensor([1.0, 3.0, 6.2831855, 100.5, 128.0, 1e-7, 1e-12, 0.3]).tolist()   # (as fp32 holds them)
    return {"plain": plain, "by parts": parts, "odd": odd}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", ["plain", "by parts", "odd"])
def test_angles(name, interleaved):
    freqs = tables()[name]
    n, N = len(freqs), len(POSITIONS)
    a = torch.tensor([[angle(p, f) for f in freqs] for p in POSITIONS], dtype=torch.float64)
    x = torch.tensor([[nearest_pair(y) for y in row] for row in a.tolist()], dtype=torch.float64)
    q = torch.zeros(1, 1, N, 64, dtype=torch.float64)
    i1 = torch.arange(n) * 2 if interleaved else torch.arange(n)
    i2 = i1 + (1 if interleaved else n)
    q[0, 0, :, i1], q[0, 0, :, i2] = x[..., 0], x[..., 1]
    qb = q.to(torch.bfloat16)
    assert torch.equal(qb.double(), q)                        # 8-bit mantissas
    want = x[..., 0] * a.cos() - x[..., 1] * a.sin()
    mag = x.abs().sum(-1)
    assert float((want.abs() / mag).max()) < 2.0 ** -7       # (a draw would give about 0.5)
    freq, pos = torch.tensor(freqs, device="cuda"), ref.ints([POSITIONS])
    tol = (2.0 ** -22.3 + 2.0 ** -22 + 2.0 ** -23) * mag + 2.0 ** -8 * want.abs()
    out, _ = fa_rope(qb.cuda(), None, freq, pos, interleaved)
    err = (out[0, 0].cpu().double()[:, i1] - want).abs()
    assert bool((err <= tol).all()), f"{float((err / mag).max()):.3e} of the pair"
    # the append form's k takes the same angles
    kc = torch.zeros(1, 1, N, 64, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    k, v = qb.cuda(), torch.zeros_like(kc)
    fa_rope_append(k.clone(), k, v, kc, vc, ref.ints([N]), freq, pos, interleaved)
    assert torch.equal(kc, out)
