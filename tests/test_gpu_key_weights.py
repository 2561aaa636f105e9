"""Accumulated attention weight per key (fa_key_weights) against 64 bits.

Bound per key, from the arithmetic: a term exp(s - lse) carries the absolute
error of its exponent, at most 2^-24 times (d products' partial sums, each
at most S = scale * max |q|.|k|; and the few roundings of values of size
S + |lse|), and ex2's 2^-22; the sum of n terms adds n 2^-24 of itself, the
final addition half a step.  Measured errors are far below it.
"""
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import (FaError, fa_device_status, fa_fwd, fa_fwd_decode, fa_key_weights,
                                      fa_key_weights_workspace_bytes)

pytestmark = pytest.mark.gpu


def lse_of(q, k, lens, causal, scale):
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    out = torch.empty(B, H, Nq, device="cuda")
    i = torch.arange(Nq, device="cuda")[:, None]
    for b in range(B):
        n = max(0, min(lens[b], Nk))
        j = torch.arange(n, device="cuda")
        for h in range(H):
            t = q[b, h].double() @ k[b, h * Hkv // H, :n].double().T * scale
            if causal:
                t = t.masked_fill(j > n - Nq + i, -math.inf)
            out[b, h] = torch.logsumexp(t, -1) if n else -math.inf
    return out


def check(q, k, lse, w_in, w, lens, causal, scale, what):
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    G = H // Hkv
    for b in range(B):
        n = max(0, min(lens[b], Nk))
        for hk in range(Hkv):
            sl = slice(hk * G, hk * G + G)
            want = ref.key_weights(q[b, sl], k[b, hk], lse[b, sl], n, causal, scale)
            before = torch.zeros(Nk, device="cuda") if w_in is None else w_in[b, hk]
            on = torch.isfinite(lse[b, sl])
            big = 0.0
            if n and bool(on.any()):
                big = abs(scale) * float((q[b, sl][on].double().abs() @ k[b, hk, :n].double().abs().T).max()) + float(
                    lse[b, sl][on].abs().max())
            eps = 2.0 ** -24 * ((d + 6) * big + 8 + min(G * Nq, 4096))
            total = before.double() + want
            err = (w[b, hk].double() - total).abs()
            tol = eps * want + 2.0 ** -23 * total.abs() + 1e-37
            assert bool((err <= tol).all()), f"{what} b{b} hk{hk}: {float((err - tol).max()):.3e} over"
            assert torch.equal(w[b, hk, n:], before[n:]), f"{what}: rows behind the last"


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,layout", [
    (1, 1, 1, 1, 1, 64, "bhnd"),
    (3, 2, 2, 1, 300, 128, "bhnd"),
    (4, 8, 1, 3, 1025, 64, "bnhd"),
    (2, 8, 2, 33, 700, 128, "pitch"),
    (2, 4, 2, 130, 513, 64, "bhnd"),
    (5, 4, 4, 200, 150, 128, "bnhd"),
    (1, 40, 1, 5, 260, 128, "bhnd"),
    (1, 2, 1, 1000, 1000, 128, "bhnd"),
    (2, 3, 1, 127, 2049, 64, "bhnd"),
])
def test_key_weights(B, H, Hkv, Nq, Nk, d, layout, causal):
    g = ref.gen(Nq + Nk)
    scale = 1 / math.sqrt(d)
    q, k = ref.draw(g, B, H, Nq, d, layout), ref.draw(g, B, Hkv, Nk, d, layout)
    lens = ([Nk, Nk - Nk // 3, 1, Nq // 2, 0] * B)[:B]
    lse = lse_of(q, k, lens, causal, scale)
    w_in = torch.rand(B, Hkv, Nk, generator=g, device="cuda")
    w = fa_key_weights(q, k, lse, ref.ints(lens), causal, weights_in=w_in)
    assert fa_device_status() == 0
    check(q, k, lse, w_in, w, lens, causal, scale, f"Nq{Nq} Nk{Nk} causal{int(causal)}")
    w = fa_key_weights(q, k, lse, ref.ints(lens), causal)
    check(q, k, lse, None, w, lens, causal, scale, "from zeros")
    again = w_in.clone()
    fa_key_weights(q, k, lse, ref.ints(lens), causal, weights_in=again, weights=again)
    assert torch.equal(again, fa_key_weights(q, k, lse, ref.ints(lens), causal, weights_in=w_in)), "in place"


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales(scale):
    g = ref.gen(70)
    q, k = ref.draw(g, 2, 4, 70, 128), ref.draw(g, 2, 2, 300, 128)
    lse = lse_of(q, k, [300, 300], True, scale)
    w = fa_key_weights(q, k, lse, None, True, scale)
    check(q, k, lse, None, w, [300, 300], True, scale, f"scale {scale}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [3, 150])
def test_hidden_rows_hold_anything(d, Nq):
    """NaN and infinities in padded query rows (lse = -inf) and behind the cache's end add nothing."""
    g = ref.gen(71)
    B, H, Hkv, Nk = 2, 4, 2, 300
    q, k = ref.draw(g, B, H, Nq, d), ref.draw(g, B, Hkv, Nk, d)
    lens = [290, 140]
    scale = 1 / math.sqrt(d)
    lse = lse_of(q, k, lens, False, scale)
    lse[:, :, 0] = -math.inf
    lse[1, 2, Nq // 2:] = -math.inf
    q[:, :, 0] = math.nan
    q[1, 2, Nq // 2:] = math.inf
    for b, n in enumerate(lens):
        k[b, 0, n:] = math.nan
        k[b, 1, n:] = -math.inf
    w_in = torch.rand(B, Hkv, Nk, generator=g, device="cuda")
    w = fa_key_weights(q, k, lse, ref.ints(lens), False, weights_in=w_in)
    assert fa_device_status() == 0 and bool(torch.isfinite(w).all())
    check(q, k, lse, w_in, w, lens, False, scale, "hidden")


@pytest.mark.parametrize("causal", [False, True])
def test_with_the_forward_and_decode_calls(causal):
    """The lse that fa_fwd and fa_fwd_decode return: the weights of a query row sum to one."""
    g = ref.gen(72)
    B, H, N, d = 2, 3, 500, 64
    q, k, v = (ref.draw(g, B, H, N, d) for _ in range(3))
    _, lse = fa_fwd(q, k, v, causal)
    w = fa_key_weights(q, k, lse, None, causal)
    # a term is off by at most the lse's 1e-4 relative, N rows sum to N
    assert bool(((w.double().sum(-1) - N).abs() <= 1e-4 * N).all())
    check(q, k, lse, None, w, [N] * B, causal, 1 / math.sqrt(d), "after fa_fwd")
    cl = ref.ints([500, 77])
    _, lse = fa_fwd_decode(q[:, :, :4], k, v, cl, causal)
    w = fa_key_weights(q[:, :, :4], k, lse, cl, causal)
    assert bool(((w.double().sum(-1) - 4).abs() <= 4e-4).all())


def test_long_cache_offsets_past_2_31():
    g = ref.gen(73)
    Nk, d, Nq = (1 << 24) + 77, 128, 2
    q = ref.draw(g, 1, 1, Nq, d)
    k = torch.empty(1, 1, Nk, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    assert k.numel() > 1 << 31
    k[0, 0, -60] = q[0, 0, 0] * 2
    scale = 1 / math.sqrt(d)
    t = torch.cat([q[0, 0].double() @ x.double().T * scale for x in k[0, 0].split(1 << 21)], -1)
    t[0, Nk - 1] = -math.inf
    lse = torch.logsumexp(t, -1).float()[None, None]
    w = fa_key_weights(q, k, lse, None, True)
    want = torch.where(t == -math.inf, torch.zeros_like(t), (t - lse[0, 0].double()[:, None]).exp()).sum(0)
    assert fa_device_status() == 0
    assert bool(((w[0, 0].double() - want).abs() <= 2e-5 * want + 1e-37).all())  # exponents of at most 60 * 134 * 2^-24


def test_workspace_streams_and_capture():
    g = ref.gen(74)
    B, H, Hkv, Nq, Nk, d = 1, 4, 2, 600, 700, 128
    q, k = ref.draw(g, B, H, Nq, d), ref.draw(g, B, Hkv, Nk, d)
    lse = lse_of(q, k, [Nk], True, 1 / math.sqrt(d))
    want = fa_key_weights(q, k, lse, None, True)
    need = fa_key_weights_workspace_bytes(B, H, Hkv, Nq, Nk, d)
    ws = torch.full((need + 512,), 99, device="cuda", dtype=torch.uint8)
    buf = torch.full((Hkv * Nk + 8,), 7.0, device="cuda")
    w = buf[4:-4].view(B, Hkv, Nk)
    fa_key_weights(q, k, lse, None, True, weights=w, workspace=ws[:need] if need else None)
    assert torch.equal(w, want) and bool((buf[:4] == 7).all()) and bool((buf[-4:] == 7).all())
    assert bool((ws[need:] == 99).all())
    if need:
        with pytest.raises(FaError):
            fa_key_weights(q, k, lse, None, True, workspace=ws[:need - 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = fa_key_weights(q, k, lse, None, True, stream=s)
    s.synchronize()
    assert torch.equal(a, want)
    outs, graphs = [], []
    for _ in range(2):
        outs.append(torch.zeros(B, Hkv, Nk, device="cuda"))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fa_key_weights(q, k, lse, None, True, weights_in=outs[-1], weights=outs[-1])
    for x in (0, 1, 0):
        graphs[x].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], want)
    assert torch.equal(outs[0], fa_key_weights(q, k, lse, None, True, weights_in=want))


def test_refusals():
    q = torch.zeros(1, 4, 8, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 32, 64, device="cuda", dtype=torch.bfloat16)
    lse = torch.zeros(1, 4, 8, device="cuda")
    with pytest.raises(ValueError):
        fa_key_weights(q[:, :3], k, lse[:, :3])
    with pytest.raises(ValueError):
        fa_key_weights(q, k, lse.double())
    with pytest.raises(ValueError):
        fa_key_weights(q, k, lse, weights_in=torch.zeros(1, 2, 31, device="cuda"))
    with pytest.raises(FaError):
        fa_key_weights(q, k, lse, scale=math.inf)
    w = torch.zeros(1 * 2 * 32 + 4, device="cuda")
    with pytest.raises(FaError):   # partly on weights_in
        fa_key_weights(q, k, lse, weights_in=w[:64].view(1, 2, 32), weights=w[4:].view(1, 2, 32))
