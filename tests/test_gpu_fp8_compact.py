"""Rows of a cache held in 8 bits moved together (fa_cache_compact_fp8): codes and
scales equal to the definition's to the last bit."""
import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import fa_cache_compact_fp8

pytestmark = pytest.mark.gpu


def same(got, want, what):
    got, want = got.double().cpu(), want.cpu()
    on = ~torch.isnan(want)
    assert torch.equal(got[on], want[on]), what


def check(kc, ks, ko, kso, before_o, before_so, kept, base, block, what):
    """ko, kso after the call; before_o, before_so what they held; kc, ks the source as it was."""
    B, Hkv = kc.shape[:2]
    rows = kept.tolist()
    for b in range(B):
        for h in range(Hkv):
            lst = rows[b] if kept.dim() == 2 else rows[b][h]
            want, want_s = r8.compact(kc[b, h].double().cpu(), ks[b, h].double().cpu(), before_o[b, h].double().cpu(),
                                      before_so[b, h].double().cpu(), lst, base[b], block)
            same(ko[b, h], want, f"{what} codes b{b} h{h}")
            same(kso[b, h], want_s, f"{what} scales b{b} h{h}")


def lists(g, B, Hkv, Nk, M, ragged=True):
    kept = torch.rand(B, Hkv, Nk, generator=g, device="cuda").argsort(-1)[..., :M].sort(-1)[0].to(torch.int32)
    if ragged:
        used = torch.tensor([[M - (3 * b + 5 * h) % M for h in range(Hkv)] for b in range(B)], device="cuda")
        kept = torch.where(torch.arange(M, device="cuda") < used[..., None], kept, torch.full_like(kept, -1))
    return kept


SHAPES = [(1, 1, 1, 1, 64, 16, "bhnd"), (2, 3, 100, 40, 64, 16, "bnhd"), (2, 2, 300, 130, 128, 64, "bhnd"),
          (1, 2, 1000, 513, 64, 128, "pitch"), (3, 2, 257, 257, 128, 32, "bnhd"), (1, 1, 3000, 1500, 128, 64, "bhnd")]


@pytest.mark.parametrize("B,Hkv,Nk,M,d,block,layout", SHAPES)
def test_out_of_place(B, Hkv, Nk, M, d, block, layout):
    g = ref.gen(3000 + Nk)
    kc, ks = r8.cache(g, B, Hkv, Nk, d, block, layout, 5)
    vc, vs = r8.cache(g, B, Hkv, Nk, d, block, layout, 5)
    Nout = M + 21
    ko, kso = r8.cache(g, B, Hkv, Nout, d, block, "bhnd", 5)
    vo, vso = r8.cache(g, B, Hkv, Nout, d, block, layout, 5)
    for kept in (lists(g, B, Hkv, Nk, M), lists(g, B, Hkv, Nk, M)[:, 0],
                 torch.randint(-2, Nk + 3, (B, Hkv, M), generator=g, device="cuda", dtype=torch.int32)):
        old = [t.clone() for t in (ko, kso, vo, vso)]
        out = fa_cache_compact_fp8(kc, vc, ks, vs, kept, block=block, k_out=ko, v_out=vo, k_scale_out=kso, v_scale_out=vso)
        assert out[0] is ko and out[3] is vso
        check(kc, ks, ko, kso, old[0], old[1], kept, [0] * B, block, "k")
        check(vc, vs, vo, vso, old[2], old[3], kept, [0] * B, block, "v")


@pytest.mark.parametrize("B,Hkv,Nk,M,d,block,layout", SHAPES)
def test_in_place(B, Hkv, Nk, M, d, block, layout):
    g = ref.gen(3100 + Nk)
    kc, ks = r8.cache(g, B, Hkv, Nk, d, block, layout, 5)
    vc, vs = r8.cache(g, B, Hkv, Nk, d, block, layout, 5)
    old = [t.clone() for t in (kc, ks, vc, vs)]
    kept = lists(g, B, Hkv, Nk, M)
    fa_cache_compact_fp8(kc, vc, ks, vs, kept, block=block)
    check(old[0], old[1], kc, ks, old[0], old[1], kept, [0] * B, block, "k")
    check(old[2], old[3], vc, vs, old[2], old[3], kept, [0] * B, block, "v")


@pytest.mark.parametrize("B,Hkv,Nk,M,d,block,layout", [
    (1, 2, 5000, 4000, 128, 16, "bhnd"), (1, 1, 6000, 3333, 64, 128, "bnhd"), (3, 7, 2100, 1500, 128, 32, "pitch"),
    (2, 20, 1300, 1299, 128, 64, "bhnd"), (5, 40, 700, 600, 64, 64, "bnhd")])
def test_long_lists_in_place(B, Hkv, Nk, M, d, block, layout):
    """From one head shared by a cluster to heads of their own; lists from a base on, which may leave nothing to move."""
    g = ref.gen(3150 + Nk)
    for base in (None, [(37 * b) % 300 for b in range(B)]):
        kc, ks = r8.cache(g, B, Hkv, Nk, d, block, layout, 5)
        vc, vs = r8.cache(g, B, Hkv, Nk, d, block, layout, 5)
        old = [t.clone() for t in (kc, ks, vc, vs)]
        kept = lists(g, B, Hkv, Nk, M)
        fa_cache_compact_fp8(kc, vc, ks, vs, kept, None if base is None else ref.ints(base), block)
        base = base or [0] * B
        check(old[0], old[1], kc, ks, old[0], old[1], kept, base, block, "k")
        check(old[2], old[3], vc, vs, old[2], old[3], kept, base, block, "v")


@pytest.mark.parametrize("d,block", [(64, 16), (128, 64), (64, 128), (128, 32)])
def test_accepted_branch(d, block):
    """A drafted tree's branch behind rows that stay, from every place in a block; rows out of the cache are skipped."""
    g = ref.gen(3200 + block)
    B, Hkv, Nk, Nt = 9, 2, 400, 40
    base = [0, 1, 15, 16, 63, 100, 360, 380, 399]
    kc, ks = r8.cache(g, B, Hkv, Nk, d, block, "bnhd", 6)
    vc, vs = r8.cache(g, B, Hkv, Nk, d, block, "bnhd", 6)
    branch = torch.full((B, Nt), -1, dtype=torch.int32)
    for b in range(B):
        path = sorted(torch.randperm(Nt)[:1 + 4 * b].tolist())
        branch[b, :len(path)] = torch.tensor(path)
    branch = branch.cuda()
    old = [t.clone() for t in (kc, ks, vc, vs)]
    fa_cache_compact_fp8(kc, vc, ks, vs, branch, base=ref.ints(base), block=block)
    check(old[0], old[1], kc, ks, old[0], old[1], branch, base, block, "k")
    check(old[2], old[3], vc, vs, old[2], old[3], branch, base, block, "v")
    # out of place, and from before the cache's start
    base = [-3, -50] + base[2:]
    ko, kso, vo, vso = (t.clone() for t in old)
    fa_cache_compact_fp8(old[0], old[2], old[1], old[3], branch, ref.ints(base), block, ko, vo, kso, vso)
    check(old[0], old[1], ko, kso, old[0], old[1], branch, base, block, "k out of place")
    check(old[2], old[3], vo, vso, old[2], old[3], branch, base, block, "v out of place")


def test_nothing_moves():
    g = ref.gen(3300)
    kc, ks = r8.cache(g, 2, 2, 200, 64, 32)
    vc, vs = r8.cache(g, 2, 2, 200, 64, 32)
    old = [t.clone() for t in (kc, ks, vc, vs)]
    fa_cache_compact_fp8(kc, vc, ks, vs, torch.full((2, 50), -1, dtype=torch.int32, device="cuda"), ref.ints([10, 70]), 32)
    fa_cache_compact_fp8(kc, vc, ks, vs, torch.arange(200, dtype=torch.int32, device="cuda").expand(2, 200).contiguous(), block=32)
    for x, y in zip(old, (kc, ks, vc, vs)):
        assert torch.equal(x.float(), y.float())


def test_graph_and_refusals():
    g = ref.gen(3400)
    kc, ks = r8.cache(g, 1, 2, 200, 128, 64)
    vc, vs = r8.cache(g, 1, 2, 200, 128, 64)
    ko, vo = kc[:, :, :100].clone(), vc[:, :, :100].clone()
    kso, vso = ks[..., :2].clone(), vs[..., :2].clone()
    kept = lists(g, 1, 2, 200, 100, False)
    out = dict(k_out=ko, v_out=vo, k_scale_out=kso, v_scale_out=vso)
    fa_cache_compact_fp8(kc, vc, ks, vs, kept, **out)
    want = [t.clone() for t in out.values()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa_cache_compact_fp8(kc, vc, ks, vs, kept, **out)
    for t in out.values():
        t.copy_(torch.zeros_like(t.float()))
    graph.replay()
    for x, y in zip(want, out.values()):
        assert torch.equal(x.float(), y.float())
    for bad in (dict(k_out=None), dict(k_scale_out=kso[..., :1]), dict(v_out=vo.float()), dict(v_out=vo[:, :, :99])):
        with pytest.raises((TypeError, ValueError)):
            fa_cache_compact_fp8(kc, vc, ks, vs, kept, **{**out, **bad})
    with pytest.raises(ValueError):
        fa_cache_compact_fp8(kc, vc, ks, vs, kept[:, :1], **out)
    with pytest.raises(ValueError):
        fa_cache_compact_fp8(kc, vc, ks, vs, kept, block=32, **out)
