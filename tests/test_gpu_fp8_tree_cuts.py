"""Attention over an 8-bit cache where more units (cache heads of all sequences) than runs
are attended to and a run ends inside the unit that it starts with: every row of o and
lse is written, whatever they held."""
import math

import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import fa_device_status, fa_fwd_tree_fp8
from test_gpu_fp8_tree import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Nt", [(1, 1), (4, 3), (8, 4), (4, 17)])
def test_units_cut_where_they_start(G, Nt, d):
    """160 units, the first sequence's four times as long as the others': run 0 and others start at their unit's start and
    end inside it."""
    g = ref.gen(2100 + G + Nt + d)
    B, Hkv, Nk, block = 20, 8, 8192, 64
    lens = [Nk] + [2000 - 13 * b for b in range(1, B)]
    q = ref.draw(g, B, Hkv * G, Nt, d)
    k, ks = r8.cache(g, B, Hkv, Nk, d, block, spread=1)
    v, vs = r8.cache(g, B, Hkv, Nk, d, block, spread=1)
    scale = 0.5 / math.sqrt(d)
    o = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:3], math.nan, device="cuda")
    for _ in range(20):
        o.fill_(math.nan)
        lse.fill_(math.nan)
        fa_fwd_tree_fp8(q, k, v, ks, vs, None, ref.ints(lens), scale, block, o, lse)
        assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(o).all())
    assert fa_device_status() == 0
    for b, hk in [(0, h) for h in range(Hkv)] + [(1, 0), (7, 3), (19, 7)]:
        heads = slice(hk * G, hk * G + G)
        kv, vv = (r8.values(c[b:b + 1, hk:hk + 1], s[b:b + 1, hk:hk + 1], block)[0, 0] for c, s in ((k, ks), (v, vs)))
        check(o[b, heads], lse[b, heads], q[b, heads], kv, vv, None, lens[b], Nt, scale, f"b{b} hk{hk}",
              (v[b, hk], vs[b, hk], block))
