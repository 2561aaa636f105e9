"""Blocks of an 8-bit cache that hold none but padding nodes' rows: neither their codes nor
their scales reach a result, whatever they are."""
import math

import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import fa_device_status, fa_fwd_tree_fp8, fa_rope_append_fp8, fa_rope_frequencies
from test_gpu_fp8_tree import check

pytestmark = pytest.mark.gpu


def drafts(B, Nt, used):
    """Chains of `used` nodes; the rest of the Nt is padding."""
    return ref.ints([[i - 1 if i < n else -2 for i in range(Nt)] for n in used])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("Nt,used,lens", [
    (7, [1, 3], [486, 100]),        # the padding starts with a block
    (16, [4, 16], [988, 320]),
    (40, [8, 24], [1000, 552]),     # two and a half blocks of padding
    (120, [3, 77], [4100, 120]),    # (the second sequence is all tree)
])
def test_scales_under_padding_reach_nothing(Nt, used, lens, G, d):
    """The same bits with any scale and any codes there."""
    g = ref.gen(2200 + Nt + d)
    B, Hkv, Nk, block = 2, 2, 4200, 16
    q = ref.draw(g, B, Hkv * G, Nt, d)
    k, ks = r8.cache(g, B, Hkv, Nk, d, block)
    v, vs = r8.cache(g, B, Hkv, Nk, d, block)
    par, n = drafts(B, Nt, used), ref.ints(lens)
    want = fa_fwd_tree_fp8(q, k, v, ks, vs, par, n, block=block)
    dead = []                       # blocks with padding nodes' rows only
    for b in range(B):
        first = -(-(lens[b] - Nt + used[b]) // block)
        dead.append(slice(first, -(-lens[b] // block)))
    assert dead[0].start < dead[0].stop
    for scale in (2.0 ** 120, 2.0 ** -100, math.nan, math.inf, 3e38, 0.0, -1.0):
        for code in (0x7E, 0x7F):
            for b in range(B):
                for t in (k, v):
                    t.view(torch.uint8)[b, :, dead[b].start * block:lens[b]] = code
                for s in (ks, vs):
                    s[b, :, dead[b]] = scale
            got = fa_fwd_tree_fp8(q, k, v, ks, vs, par, n, block=block)
            assert fa_device_status() == 0
            assert torch.equal(got[1], want[1]), (scale, code)
            assert torch.equal(got[0], want[0]), (scale, code)


@pytest.mark.parametrize("d", [64, 128])
def test_padding_rows_of_any_size(d):
    """Padding nodes appended with values up to bf16's greatest: the blocks that are theirs alone take scales of up to
    2^120, and the other nodes attend as ever."""
    g = ref.gen(2210 + d)
    B, Hkv, G, Nk, Nt, block = 2, 2, 2, 400, 48, 16
    q = ref.draw(g, B, Hkv * G, Nt, d)
    k, v = ref.draw(g, B, Hkv, Nt, d), ref.draw(g, B, Hkv, Nt, d)
    kc, ks = r8.cache(g, B, Hkv, Nk, d, block)
    vc, vs = r8.cache(g, B, Hkv, Nk, d, block)
    used, lens = [16, 32], [368, 176]
    for t in (k, v):
        t[0, :, 16:] = 3e38
        t[1, :, 32:] = -3e38
    freq, _ = fa_rope_frequencies(d)
    fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, ref.ints(lens), freq, block=block)
    par = drafts(B, Nt, used)
    o, lse = fa_fwd_tree_fp8(q, kc, vc, ks, vs, par, ref.ints(lens), 0.05, block)
    assert float(vs[0, 0, 21]) == 2.0 ** 120 and fa_device_status() == 0
    kv, vv = r8.values(kc, ks, block), r8.values(vc, vs, block)
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, h * G + G)
            live = used[b]          # (the bound counts every row of a tile that a node sees, so none of the padding)
            assert bool((o[b, heads, live:] == 0).all()) and bool((lse[b, heads, live:] == -math.inf).all())
            n = lens[b] - Nt + live
            check(o[b, heads, :live], lse[b, heads, :live], q[b, heads, :live], kv[b, h, :n], vv[b, h, :n], None, n, live,
                  0.05, f"b{b} h{h}", (vc[b, h, :n], vs[b, h], block))
