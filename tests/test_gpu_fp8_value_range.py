"""Attention over an 8-bit cache whose value scales lie anywhere between 2^-100 and 2^120:
results as the 64-bit attention of the values, wherever those fit bf16."""
import math

import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import fa_device_status, fa_fwd_tree_fp8
from test_gpu_fp8_tree import check

pytestmark = pytest.mark.gpu

# rows a cache head of every kernel; one unit cut into many runs, whole units, units cut into a few
SHAPES = [(1, 1, 1, 30000), (1, 3, 3, 900), (3, 8, 2, 2500), (2, 4, 8, 3000), (1, 8, 16, 9000), (2, 2, 33, 1000)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [-90, -40, 60, 100, 116])
def test_scales_far_from_one(e, d):
    """The values of ordinary caches times 2^e."""
    for B, G, Nt, Nk in SHAPES:
        g = ref.gen(2300 + Nk)
        q = ref.draw(g, B, 2 * G, Nt, d)
        k, ks = r8.cache(g, B, 2, Nk, d, 32)
        v, vs = r8.cache(g, B, 2, Nk, d, 32, spread=1)
        vs *= 2.0 ** e
        scale = 0.7 / math.sqrt(d)
        o, lse = fa_fwd_tree_fp8(q, k, v, ks, vs, scale=scale, block=32)
        assert fa_device_status() == 0
        kv, vv = r8.values(k, ks, 32), r8.values(v, vs, 32)
        for b in range(B):
            check(o[b, :G], lse[b, :G], q[b, :G], kv[b, 0], vv[b, 0], None, Nk, Nt, scale, f"b{b} {G} {Nt} {Nk}",
                  (v[b, 0], vs[b, 0], 32))


@pytest.mark.parametrize("d", [64, 128])
def test_greatest_values(d):
    """All values 1.75 * 2^127, close to bf16's greatest, and their negatives: o is that value, to the weights' rounding
    (2^-9 of each or, of 128 keys each, 2^-18 of the greatest, while the sum that divides takes them unrounded) and bf16's 2^-8:
    below 2^-7 of it in all."""
    for B, G, Nt, Nk in SHAPES:
        g = ref.gen(2310 + Nk)
        q = ref.draw(g, B, 2 * G, Nt, d)
        k, ks = r8.cache(g, B, 2, Nk, d, 64)
        v = torch.full((B, 2, Nk, d), 448.0, device="cuda").to(r8.E4M3)
        v[:, 1] = (-v[:, 1].float()).to(r8.E4M3)
        vs = torch.full((B, 2, -(-Nk // 64)), 2.0 ** 119, device="cuda")
        o, lse = fa_fwd_tree_fp8(q, k, v, ks, vs)
        assert fa_device_status() == 0
        most = 448.0 * 2.0 ** 119
        want = torch.tensor([most, -most], dtype=torch.float64, device="cuda")[None, :, None, None, None]
        off = (o.double().view(B, 2, G, Nt, d) / want - 1.0).abs()
        assert float(off.max()) <= 2.0 ** -7, (G, Nt, Nk, float(off.max()))


@pytest.mark.parametrize("d", [64, 128])
def test_tiles_of_different_size(d):
    """Value scales that differ by up to 2^80 from block to block, within a tile and from tile to tile."""
    for B, G, Nt, Nk in SHAPES:
        g = ref.gen(2320 + Nk)
        q = ref.draw(g, B, 2 * G, Nt, d)
        k, ks = r8.cache(g, B, 2, Nk, d, 16)
        v, vs = r8.cache(g, B, 2, Nk, d, 16, spread=40)
        tile = torch.randint(-40, 41, (B, 2, -(-Nk // 128)), generator=g, device="cuda").repeat_interleave(8, -1)
        for s in (vs, vs * torch.exp2(tile[..., :vs.shape[-1]].float()).clamp(2.0 ** -40, 2.0 ** 40)):
            scale = 0.7 / math.sqrt(d)
            o, lse = fa_fwd_tree_fp8(q, k, v, ks, s, scale=scale, block=16)
            assert fa_device_status() == 0
            kv, vv = r8.values(k, ks, 16), r8.values(v, s, 16)
            for b in range(B):
                check(o[b, :G], lse[b, :G], q[b, :G], kv[b, 0], vv[b, 0], None, Nk, Nt, scale, f"b{b} {G} {Nt} {Nk}",
                      (v[b, 0], s[b, 0], 16))
