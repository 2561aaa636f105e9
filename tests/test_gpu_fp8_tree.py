"""Attention over a cache held in 8 bits (fa_fwd_tree_fp8) against the 64-bit
attention of the values that its codes stand for.

Bounds.  q enters as the sum of two e4m3 parts of a row scaled to at most 448 and more
than 224, off by at most 2^-10 there (the second part's least half step; bf16's
8 bits are otherwise 4 + 4), 2^-17.8 of the row's greatest value: a score is off by
that times scale * sum |k|.  It is a sum of 2 d products, exact in fp32, added in fp32 in
an order of the hardware's: off by at most 2 d * 2^-23 of scale * sum |q k| (A below;
each addition by at most 2^-23 of the running sum of magnitudes, truncation
included), then a few 2^-24 of itself, which A exceeds too: e is the sum of both.
Every weight is off by e and by the exponential's 2^-22, then by its rounding to two e4m3
parts: the first leaves at most half a step, 2^(a - 4) of a weight in
[2^a, 2^(a + 1)), and the second at most a sixteenth of a power of two below that, 2^(a - 9),
or 2^-10 where it falls below e4m3's normal range: 2^-9 of the weight, or 2^-10 with the
tile's greatest product of a weight and its value's scale at 2^8, so 2^-18 of that times
sum |codes| of the tile (F below).  O, a quotient of two sums with errors of e and 2^-22 of
their terms, is off by twice those of sum P|v| and by the roundings; then it is rounded
to bf16, 2^-8 of it.  The logsumexp takes unrounded weights: e and 2^-20 (of its sum and
its logarithm).
"""
import math

import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import (FaError, fa_device_status, fa_fwd_tree, fa_fwd_tree_fp8,
                                      fa_tree_fp8_workspace_bytes)

pytestmark = pytest.mark.gpu


def floor_of(q, kv, mask, lse, scale, vcodes, vs, block):
    """F: 2^-18 of each 128-row tile's greatest P vs, times its sum of |codes|."""
    Nk = kv.shape[0]
    s = vs.double().repeat_interleave(block)[:Nk]
    on = mask.to(q.device)
    t = q.double() @ torch.where(on.any(0)[:, None], kv, torch.zeros_like(kv)).T * scale
    p = torch.where(on, (t - lse[:, None].clamp(min=-1e30)).exp() * s.nan_to_num(), torch.zeros_like(t))
    c = torch.where(on.any(0)[:, None], vcodes.double().abs().nan_to_num(), torch.zeros_like(kv))
    pad = -Nk % 128
    p = torch.nn.functional.pad(p, (0, pad)).view(p.shape[0], -1, 128).amax(-1)
    c = torch.nn.functional.pad(c, (0, 0, 0, pad)).view(-1, 128, c.shape[1]).sum(1)
    return 2.0 ** -18 * p @ c


def check(o, lse, q, kv, vv, parents, n, Nt, scale, what, v8):
    """One (b, hk): q [G, Nt, d], values kv, vv [Nk, d]; parents a list or None; v8: V's codes, scales and block."""
    Nk, d = kv.shape
    par = list(range(-1, Nt - 1)) if parents is None else parents
    mask = ref.tree_mask(par, n, Nt, Nk)
    on = mask.any(1).to(q.device)
    for h in range(q.shape[0]):
        wo, wl, pv, A = r8.attention(q[h], kv, vv, mask, scale)
        e = (2 * d + 8) * 2.0 ** -23 * A
        e += 2.0 ** -17.8 * float(q[h].abs().max()) * float(kv[mask.any(0).to(kv.device)].abs().sum(-1).max().nan_to_num()
                                                            if bool(mask.any()) else 0.0) * abs(scale)
        assert bool((lse[h][~on] == -math.inf).all()) and bool((o[h][~on] == 0).all()), what
        err = (o[h].double() - wo).abs()[on]
        tol = (4 * e + 2.0 ** -21 + 2.0 ** -9) * pv[on] + floor_of(q[h], kv, mask, wl, scale, *v8)[on]
        tol += 2.0 ** -8 * wo.abs()[on] + 1e-30
        assert bool((err <= tol).all()), f"{what} head {h}: {float(err.max()):.3e}, {float((err / tol).max()):.2f} of the bound"
        err = (lse[h].double() - wl).abs()[on]
        assert bool((err <= e + 2.0 ** -20 * (1 + wl[on].abs())).all()), f"{what} head {h}: lse {float(err.max()):.3e}"


def tree_of(g, B, Nt):
    i = torch.arange(Nt, device="cuda")
    u = torch.rand(B, Nt, generator=g, device="cuda")
    return (torch.minimum((u * (i + 1)).floor(), i.float()) - 1).to(torch.int32)


def run(g, B, H, Hkv, Nt, Nk, d, block, layout="bhnd", lens=None, parents=None, scale=None, spread=3, mult=1.0, heads=None):
    G = H // Hkv
    q = ref.draw(g, B, H, Nt, d, layout if layout != "pitch" else "bhnd", mult)
    k, ks = r8.cache(g, B, Hkv, Nk, d, block, layout, spread)
    v, vs = r8.cache(g, B, Hkv, Nk, d, block, layout, spread)
    s = scale if scale is not None else 0.7 / math.sqrt(d) / 2 ** spread
    o, lse = fa_fwd_tree_fp8(q, k, v, ks, vs, parents, None if lens is None else ref.ints(lens), s, block)
    assert fa_device_status() == 0
    kv, vv = r8.values(k, ks, block), r8.values(v, vs, block)
    for b in range(B):
        for hk in range(Hkv):
            if heads is not None and (b, hk) not in heads:
                continue
            par = None if parents is None else parents[b].tolist() if parents.dim() == 2 else parents.tolist()
            check(o[b, hk * G:hk * G + G], lse[b, hk * G:hk * G + G], q[b, hk * G:hk * G + G], kv[b, hk], vv[b, hk], par,
                  Nk if lens is None else lens[b], Nt, s, f"b{b} hk{hk}", (v[b, hk], vs[b, hk], block))
    return o, lse


@pytest.mark.parametrize("B,H,Hkv,Nt,Nk,d,block,layout", [
    (1, 1, 1, 1, 1, 64, 16, "bhnd"),
    (1, 1, 1, 1, 1, 128, 128, "bhnd"),
    (2, 4, 2, 1, 129, 64, 32, "bnhd"),
    (2, 4, 2, 1, 1000, 128, 64, "bhnd"),
    (1, 8, 1, 1, 5000, 128, 16, "pitch"),
    (1, 8, 1, 1, 5000, 64, 128, "pitch"),
    (3, 6, 6, 3, 700, 64, 64, "bhnd"),
    (2, 16, 2, 2, 3001, 128, 32, "bnhd"),      # 16 rows a cache head
    (2, 17, 1, 1, 2100, 128, 64, "bhnd"),      # 17
    (1, 8, 2, 8, 2500, 64, 64, "bhnd"),        # 32
    (1, 4, 1, 9, 2500, 128, 64, "bhnd"),       # 36
    (1, 8, 1, 8, 1500, 64, 16, "bnhd"),        # 64
    (1, 4, 2, 33, 3000, 128, 128, "bhnd"),     # 66
    (1, 2, 2, 128, 2000, 64, 64, "bhnd"),      # 128
    (1, 3, 1, 64, 1100, 128, 32, "bhnd"),      # 192 rows: two groups
    (1, 16, 1, 128, 1300, 64, 64, "bhnd"),     # 2048 rows: 16 groups
])
def test_shapes(B, H, Hkv, Nt, Nk, d, block, layout):
    g = ref.gen(2000 + Nk + Nt)
    run(g, B, H, Hkv, Nt, Nk, d, block, layout)
    lens = [min(Nk, max(Nt, Nk - 37 * b - Nk // 3)) for b in range(B)]
    run(g, B, H, Hkv, Nt, Nk, d, block, layout, lens, tree_of(g, B, Nt))


def test_long_and_many_units():
    g = ref.gen(2001)
    run(g, 1, 4, 1, 1, 100001, 128, 64)                                        # one unit cut into all runs
    run(g, 1, 2, 1, 5, 70000, 64, 16, "bnhd")
    run(g, 40, 8, 4, 2, 1500, 64, 32, lens=[1500 - 31 * b for b in range(40)], heads=[(b, b % 4) for b in range(0, 40, 3)])
    run(g, 200, 2, 1, 1, 400, 128, 64, lens=[(b * 7) % 400 + 1 for b in range(200)], heads=[(b, 0) for b in range(0, 200, 11)])


@pytest.mark.parametrize("d,H,Nt", [(64, 2, 1), (128, 4, 3), (128, 20, 2)])
def test_more_sequences_than_threads(d, H, Nt):
    g = ref.gen(2030 + d + H)
    lens = [(b * 37) % 140 for b in range(3001)]
    run(g, 3001, H, 1, Nt, 139, d, 32, lens=lens, heads=[(b, 0) for b in list(range(0, 3001, 250)) + [1, 2, 3, 2999, 3000]])


def test_k_and_v_laid_out_differently():
    """Strides of their own for q, k, v and o, scales apart: the same bits as packed tensors."""
    g = ref.gen(2031)
    for d, G, Nt in ((64, 2, 3), (128, 3, 7), (128, 8, 9)):
        q = ref.draw(g, 2, 2 * G, Nt, d, "bnhd")
        k, ks = r8.cache(g, 2, 2, 1300, d, 32, "bnhd")
        v, vs = r8.cache(g, 2, 2, 1300, d, 32, "pitch")
        o = torch.zeros(2, Nt, 2 * G, d + 8, device="cuda", dtype=torch.bfloat16).transpose(1, 2)[..., :d]
        par, lens = tree_of(g, 2, Nt), ref.ints([1300, 900])
        want = fa_fwd_tree_fp8(q.contiguous(), k.contiguous(), v.contiguous(), ks, vs, par, lens, block=32)
        got = fa_fwd_tree_fp8(q, k, v, ks, vs, par, lens, block=32, o=o)
        assert got[0] is o and torch.equal(o, want[0]) and torch.equal(got[1], want[1])
        assert not bool(o.as_strided((2, Nt, 2 * G, 8), (Nt * 2 * G * (d + 8), 2 * G * (d + 8), d + 8, 1), d).any())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Nt", [(8, 1), (3, 3), (1, 7), (4, 4), (17, 1), (2, 16), (1, 33), (4, 16), (5, 13), (2, 64), (43, 3), (8, 40)])
def test_rows_of_a_group(G, Nt, d):
    """Query rows of a cache head around the kernels' 8, 16, 32 and 128, over caches whose units are cut by the runs' ends,
    and of which a run holds several."""
    g = ref.gen(2020 + G + Nt)
    run(g, 3, 5 * G, 5, Nt, 2900, d, 64, "bnhd", [2900, 2000, 1300], tree_of(g, 3, Nt), heads=[(0, 0), (0, 4), (1, 2), (2, 0)])
    lens = [1100 - 29 * b for b in range(36)]
    run(g, 36, 8 * G, 8, Nt, 1100, d, 32, lens=lens, heads=[(0, 0), (1, 7), (9, 3), (20, 5), (35, 7)])
    run(g, 36, 2 * G, 2, Nt, 500, d, 16, lens=[n % 501 for n in lens], heads=[(0, 0), (1, 1), (9, 0), (20, 1), (35, 1)])


@pytest.mark.parametrize("d", [64, 128])
def test_lengths(d):
    """Every residue of the length against slices and tiles; lengths of zero, below Nt, negative, past Nk."""
    g = ref.gen(2002)
    Nk, Nt = 300, 3
    lens = [0, 1, 2, 3, 15, 16, 17, 18, 19, 31, 32, 33, 127, 128, 129, 130, 131, 143, 144, 255, 256, 257, 299, 300, 301, -5, 99999]
    for parents in (None, ref.ints([-1, 0, 0])):
        run(g, len(lens), 2, 1, Nt, Nk, d, 16, lens=lens, parents=parents)
    for H, Nt in ((2, 12), (3, 25)):
        run(g, len(lens), H, 1, Nt, Nk, d, 64, lens=lens, parents=tree_of(g, len(lens), Nt))


def test_padding_and_invalid_parents():
    g = ref.gen(2003)
    par = ref.ints([[-1, 0, 1, -2, 3, 4, 9, 1, -1, 5], [-1, -1, -1, 2, 2, 2, 3, 7, 0, 8], [-2] + [0] * 9, [1] + [-1] * 9])
    run(g, 4, 6, 2, 10, 500, 64, 32, lens=[500, 300, 200, 140], parents=par)
    run(g, 4, 6, 2, 10, 2990, 128, 64, lens=[2990, 2900, 2000, 140], parents=par)
    run(g, 4, 10, 2, 10, 2990, 128, 64, lens=[2990, 2900, 2000, 140], parents=par)
    run(g, 4, 10, 2, 10, 700, 64, 16, lens=[700, 640, 500, 140], parents=par)


def test_chain_is_the_causal_tree():
    g = ref.gen(2004)
    q = ref.draw(g, 2, 4, 40, 128)
    k, ks = r8.cache(g, 2, 2, 900, 128, 64)
    v, vs = r8.cache(g, 2, 2, 900, 128, 64)
    a = fa_fwd_tree_fp8(q, k, v, ks, vs, None, ref.ints([900, 20]))
    z = fa_fwd_tree_fp8(q, k, v, ks, vs, ref.ints(list(range(-1, 39))), ref.ints([900, 20]))
    assert torch.equal(a[0], z[0]) and torch.equal(a[1], z[1])


def test_against_the_bf16_tree():
    """Codes that bf16 holds: the same attention as fa_fwd_tree's of their values, within both roundings."""
    g = ref.gen(2005)
    q = ref.draw(g, 2, 8, 12, 128)
    k, ks = r8.cache(g, 2, 2, 2000, 128, 64, spread=1)
    v, vs = r8.cache(g, 2, 2, 2000, 128, 64, spread=1)
    par = tree_of(g, 2, 12)
    o, lse = fa_fwd_tree_fp8(q, k, v, ks, vs, par)
    o2, lse2 = fa_fwd_tree(q, r8.values(k, ks, 64).to(torch.bfloat16), r8.values(v, vs, 64).to(torch.bfloat16), par)
    on = torch.isfinite(lse)
    assert torch.equal(on, torch.isfinite(lse2)) and float((lse - lse2).abs()[on].max()) < 1e-4
    assert float((o.double() - o2.double()).abs().max()) < 2.0 ** -7 * float(o.abs().max()) + 2.0 ** -8


@pytest.mark.parametrize("mult,scale", [(1.0, 0.0), (1.0, -0.05), (30.0, 0.2), (1e-4, 300.0), (1.0, 3e-3)])
def test_scales_and_sharp_rows(mult, scale):
    g = ref.gen(2006)
    run(g, 2, 4, 2, 5, 1500, 64, 32, scale=scale, mult=mult, parents=tree_of(g, 2, 5))
    run(g, 1, 4, 2, 20, 1500, 128, 64, scale=scale, mult=mult)


def test_scales_far_apart():
    """Neighbouring blocks whose scales differ by up to 2^16, V's and K's, in every order."""
    g = ref.gen(2007)
    run(g, 2, 4, 2, 2, 2000, 128, 16, spread=8, scale=1e-4)
    run(g, 2, 4, 2, 2, 2000, 64, 128, spread=8, scale=1e-4)


def test_tiny_and_huge_q():
    """bf16's range in q: rows of 2^-120 and 2^120 with scales to match; zeros."""
    g = ref.gen(2008)
    q = ref.draw(g, 1, 4, 1, 128)
    k, ks = r8.cache(g, 1, 1, 500, 128, 64)
    v, vs = r8.cache(g, 1, 1, 500, 128, 64)
    want = fa_fwd_tree_fp8(q, k, v, ks, vs, scale=0.01)
    for e in (-90, 90):
        got = fa_fwd_tree_fp8(q * 2.0 ** e, k, v, ks, vs, scale=0.01 * 2.0 ** -e)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    o, lse = fa_fwd_tree_fp8(torch.zeros_like(q), k, v, ks, vs)
    assert float((lse - math.log(500)).abs().max()) < 1e-5
    mean = r8.values(v, vs, 64)[0, 0].mean(0)
    assert float((o[0, :, 0].double() - mean).abs().max()) <= 2.0 ** -8 * float(mean.abs().max()) + 1e-4


def test_garbage_behind_the_rows_and_under_padding():
    """NaN codes and NaN scales behind the last row, and NaN codes in padding nodes' rows, reach nothing."""
    g = ref.gen(2009)
    for Nk, n, d in ((600, 333, 64), (5000, 4010, 128), (3000, 2048, 128)):
        q = ref.draw(g, 1, 4, 6, d)
        k, ks = r8.cache(g, 1, 2, Nk, d, 32)
        v, vs = r8.cache(g, 1, 2, Nk, d, 32)
        par = ref.ints([-1, 0, -2, 1, 2, 0])
        want = fa_fwd_tree_fp8(q, k, v, ks, vs, par, ref.ints([n]), block=32)
        for t in (k, v):
            raw = t.view(torch.uint8)
            raw[:, :, n:] = 0x7F
            raw[:, :, n - 4] = 0xFF   # node 2 and node 4, below it
            raw[:, :, n - 2] = 0x7F
        for s in (ks, vs):
            s[..., -(-n // 32):] = math.nan
        got = fa_fwd_tree_fp8(q, k, v, ks, vs, par, ref.ints([n]), block=32)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert bool(torch.isfinite(got[0]).all())


def test_nan_reaches_its_rows():
    """A NaN key makes the rows that see it NaN, and no other; so does a NaN query row."""
    g = ref.gen(2010)
    for Nk in (400, 4000):
        q = ref.draw(g, 1, 2, 4, 64)
        k, ks = r8.cache(g, 1, 1, Nk, 64, 16)
        v, vs = r8.cache(g, 1, 1, Nk, 64, 16)
        par = ref.ints([-1, 0, 0, 1])
        clean = fa_fwd_tree_fp8(q, k, v, ks, vs, par, block=16)
        bad = k.clone()
        bad.view(torch.uint8)[0, 0, Nk - 3, 5] = 0x7F   # node 1: seen by nodes 1 and 3
        o, lse = fa_fwd_tree_fp8(q, bad, v, ks, vs, par, block=16)
        assert bool(torch.isnan(o[0, :, [1, 3]]).all()) and bool(torch.isnan(lse[0, :, [1, 3]]).all())
        assert torch.equal(o[0, :, [0, 2]], clean[0][0, :, [0, 2]]) and torch.equal(lse[0, :, [0, 2]], clean[1][0, :, [0, 2]])
        bad = k.clone()
        bad.view(torch.uint8)[0, 0, 7, 5] = 0x7F
        o, lse = fa_fwd_tree_fp8(q, bad, v, ks, vs, par, block=16)
        assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
        qn = q.clone()
        qn[0, 1, 2, 9] = math.nan
        o, lse = fa_fwd_tree_fp8(qn, k, v, ks, vs, par, block=16)
        assert bool(torch.isnan(o[0, 1, 2]).all()) and bool(torch.isnan(lse[0, 1, 2]))
        assert torch.equal(o[0, 0], clean[0][0, 0]) and torch.equal(o[0, 1, :2], clean[0][0, 1, :2])
        bad = v.clone()
        bad.view(torch.uint8)[0, 0, 7, 5] = 0x7F
        o, lse = fa_fwd_tree_fp8(q, k, bad, ks, vs, par, block=16)
        assert bool(torch.isnan(o[..., 5]).all()) and torch.equal(lse, clean[1])
        assert torch.equal(o[..., :5], clean[0][..., :5]) and torch.equal(o[..., 6:], clean[0][..., 6:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [5, 12])
def test_nan_and_many_rows(G, d):
    """The same for the other kernels: NaN keys and queries reach the rows that see them, garbage behind none."""
    g = ref.gen(2021)
    Nk, n = 2500, 2222
    q = ref.draw(g, 1, 2 * G, 4, d)
    k, ks = r8.cache(g, 1, 2, Nk, d, 16)
    v, vs = r8.cache(g, 1, 2, Nk, d, 16)
    par, lens = ref.ints([-1, 0, 0, 1]), ref.ints([n])
    clean = fa_fwd_tree_fp8(q, k, v, ks, vs, par, lens, block=16)
    for t in (k, v):
        t.view(torch.uint8)[:, :, n:] = 0x7F
    ks[..., -(-n // 16):] = math.nan
    vs[..., -(-n // 16):] = math.inf
    o, lse = fa_fwd_tree_fp8(q, k, v, ks, vs, par, lens, block=16)
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1]) and bool(torch.isfinite(o).all())
    bad = k.clone()
    bad.view(torch.uint8)[0, 0, n - 3, 5] = 0x7F    # node 1: seen by nodes 1 and 3
    o, lse = fa_fwd_tree_fp8(q, bad, v, ks, vs, par, lens, block=16)
    assert bool(torch.isnan(o[0, :G, [1, 3]]).all()) and bool(torch.isnan(lse[0, :G, [1, 3]]).all())
    assert torch.equal(o[0, :G, [0, 2]], clean[0][0, :G, [0, 2]]) and torch.equal(lse[0, :G, [0, 2]], clean[1][0, :G, [0, 2]])
    assert torch.equal(o[0, G:], clean[0][0, G:])
    qn = q.clone()
    qn[0, 1, 2, 9] = math.inf
    o, lse = fa_fwd_tree_fp8(qn, k, v, ks, vs, par, lens, block=16)
    assert bool(torch.isnan(o[0, 1, 2]).all()) and bool(torch.isnan(lse[0, 1, 2]))
    o[0, 1, 2], lse[0, 1, 2] = clean[0][0, 1, 2], clean[1][0, 1, 2]
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


def test_same_bits_again_graphs_and_streams():
    g = ref.gen(2011)
    q = ref.draw(g, 2, 8, 4, 128)
    k, ks = r8.cache(g, 2, 2, 6000, 128, 64)
    v, vs = r8.cache(g, 2, 2, 6000, 128, 64)
    lens = ref.ints([6000, 4100])
    want = fa_fwd_tree_fp8(q, k, v, ks, vs, None, lens)
    need = fa_tree_fp8_workspace_bytes(2, 8, 2, 4, 6000, 128)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xff)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(), dict(workspace=ws), dict(stream=side)):
        got = fa_fwd_tree_fp8(q, k, v, ks, vs, None, lens, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(fa_fwd_tree_fp8(q, k, v, ks, vs, None, lens))
    for _ in range(3):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for got in outs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(FaError):
        fa_fwd_tree_fp8(q, k, v, ks, vs, None, lens, workspace=ws[:need - 256])


def test_refusals_of_the_binding():
    g = ref.gen(2012)
    q = ref.draw(g, 1, 4, 2, 64)
    k, ks = r8.cache(g, 1, 2, 100, 64, 64)
    v, vs = r8.cache(g, 1, 2, 100, 64, 64)
    for bad in (dict(q=q.float()), dict(k=k.float()), dict(k=k.view(torch.uint8)), dict(v=v[:, :, :99]), dict(ks=ks[..., :1]),
                dict(vs=vs.double()), dict(block=32), dict(block=65), dict(parents=ref.ints([0])), dict(k=k.cpu()),
                dict(cache_seqlens=ref.ints([1, 2])), dict(o=q.float()), dict(lse=torch.zeros(1, 4, 3, device="cuda"))):
        a = dict(q=q, k=k, v=v, ks=ks, vs=vs)
        a.update({x: bad[x] for x in bad if x in a})
        with pytest.raises((TypeError, ValueError)):
            fa_fwd_tree_fp8(a["q"], a["k"], a["v"], a["ks"], a["vs"], **{x: bad[x] for x in bad if x not in a})
