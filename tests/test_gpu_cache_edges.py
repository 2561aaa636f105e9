"""The cache operators where their calls meet: several at once, unusual head
counts and lists, padding in the queries.  Bounds as in the operators' own
tests, whose checks are used here."""
import math
import threading

import pytest
import torch

import cache_refs as ref
import test_gpu_key_weights as kw
import test_gpu_tree as tree
from exact_attention_48_gb300 import (fa_cache_compact, fa_cache_select, fa_device_status, fa_fwd_tree,
                                      fa_key_weights, fa_rope, fa_rope_append, fa_rope_frequencies)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nt", [24, 48])
def test_padding_nodes_queries_hold_anything(d, Nt):
    """NaN and infinities in padding nodes' query rows, one row tile and two, a cut cache and a short one."""
    g = ref.gen(90 + Nt)
    for Nk in (200, 3001):
        B, H, Hkv = 2, 8, 2
        q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
        par = tree.trees(g, B, Nt)
        lens = [Nk, Nk - 77]
        for b in range(B):
            live = ref.tree_mask(par[b].tolist(), lens[b], Nt, Nk).any(1).cuda()
            q[b, ::2, ~live] = math.nan
            q[b, 1::2, ~live] = math.inf
        o, lse = fa_fwd_tree(q, k, v, par, ref.ints(lens))
        assert fa_device_status() == 0 and bool(torch.isfinite(o).all())
        tree.check(q, k, v, par, lens, o, lse, 1 / math.sqrt(d), f"Nk{Nk}")


@pytest.mark.parametrize("H,Nt,Nk", [(310, 128, 200), (33, 128, 3001), (200, 1, 700)])
def test_tree_many_heads_share_one(H, Nt, Nk):
    """More row tiles than the GPU has multiprocessors, and a row tile count that leaves one alone."""
    g = ref.gen(91 + H)
    q, k, v = ref.draw(g, 1, H, Nt, 64), ref.draw(g, 1, 1, Nk, 64), ref.draw(g, 1, 1, Nk, 64)
    par = tree.trees(g, 1, Nt)
    o, lse = fa_fwd_tree(q, k, v, par, ref.ints([Nk - 1]))
    assert fa_device_status() == 0
    heads = [0, 1, 2, 3, H // 2, H - 2, H - 1]
    tree.check(q[:, heads], k, v, par, [Nk - 1], o[:, heads], lse[:, heads], 0.125, f"H{H}")
    again = fa_fwd_tree(q[:, 1:], k, v, par, ref.ints([Nk - 1]))
    for x in range(H - 1):   # a head's rows do not depend on their place among the others beyond rounding
        assert float((again[1][0, x] - lse[0, x + 1])[torch.isfinite(lse[0, x + 1])].abs().max()) <= 2e-4


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk", [(1, 64, 1, 1, 600), (1, 300, 1, 1, 600), (1, 128, 1, 3, 257), (700, 1, 1, 1, 5),
                                           (2, 2, 2, 64, 64), (1, 1, 1, 65, 40), (1, 1, 1, 129, 1)])
def test_key_weights_head_counts_and_short_caches(B, H, Hkv, Nq, Nk):
    g = ref.gen(92 + H + Nk)
    d = 64
    q, k = ref.draw(g, B, H, Nq, d), ref.draw(g, B, Hkv, Nk, d)
    lens = [max(0, Nk - b % 6) for b in range(B)]
    for causal in (False, True):
        lse = kw.lse_of(q, k, lens, causal, 0.125)
        w = fa_key_weights(q, k, lse, ref.ints(lens), causal)
        assert fa_device_status() == 0
        kw.check(q, k, lse, None, w, lens, causal, 0.125, f"H{H} Nq{Nq} Nk{Nk} causal{int(causal)}")


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_key_weights_scales_of_few_rows(scale):
    g = ref.gen(93)
    q, k = ref.draw(g, 2, 4, 3, 128), ref.draw(g, 2, 2, 300, 128)
    lse = kw.lse_of(q, k, [300, 300], True, scale)
    w = fa_key_weights(q, k, lse, None, True, scale)
    kw.check(q, k, lse, None, w, [300, 300], True, scale, f"scale {scale}")


def test_select_short_sequences_in_a_long_cache():
    """Lists that the cache's size cuts over a cluster, of sequences that need a part of it or nothing."""
    g = ref.gen(94)
    w = torch.rand(4, 1, 70000, generator=g, device="cuda")
    lens, keep, first, recent = [70000, 12400, 12346, 3], 12345, 5, 1000
    kept, new = fa_cache_select(w, keep, ref.ints(lens), first, recent)
    assert new.tolist() == [min(n, keep) for n in lens]
    got, cpu = kept.tolist(), w.cpu()
    for b in range(4):
        assert got[b][0] == ref.select(cpu[b, 0], lens[b], keep, first, recent), b


def test_compact_rows_named_more_than_once():
    """Out of place a list may repeat rows and be longer than either cache; shared by the batch, or by all."""
    g = ref.gen(95)
    B, Hkv, Nk, Nout, M, d = 2, 3, 50, 70, 200, 64
    k, v = ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d, "bnhd")
    w = torch.rand(B, Hkv, Nk, generator=g, device="cuda")
    lists = torch.randint(0, Nk, (B, Hkv, M), generator=g, device="cuda", dtype=torch.int32)
    for kept in (lists, lists[:, 0], lists[:1, :1].expand(B, Hkv, M), lists[0, 0].expand(B, M)):
        ko, vo = (torch.full((B, Hkv, Nout, d), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        wo = torch.full((B, Hkv, Nout), 5.0, device="cuda")
        fa_cache_compact(k, v, kept, w, None, ko, vo, wo)
        rows = (kept if kept.dim() == 3 else kept[:, None].expand(B, Hkv, M))[..., :Nout].long()
        for x, y in ((k, ko), (v, vo)):
            assert torch.equal(y, x.gather(2, rows[..., None].expand(B, Hkv, Nout, d)))
        assert torch.equal(wo, w.gather(2, rows))


def test_two_threads_on_two_streams():
    """Every operator called by two host threads at once, each on a stream of its own: the results of one thread."""
    g = ref.gen(96)
    B, H, Hkv, N, Nk, d = 2, 8, 2, 6, 2600, 128
    freq, _ = fa_rope_frequencies(d)
    par, lens = tree.trees(g, B, N), ref.ints([2600, 1234])
    sets = []
    for _ in range(2):
        sets.append((ref.draw(g, B, H, N, d), ref.draw(g, B, Hkv, N, d), ref.draw(g, B, Hkv, N, d),
                     ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)))

    def step(s):
        q, k, v, kc, vc = s[0], s[1], s[2], s[3].clone(), s[4].clone()
        a, b = fa_rope(q, k, freq)
        qr = fa_rope_append(q, k, v, kc, vc, lens, freq)
        o, lse = fa_fwd_tree(qr, kc, vc, par, lens)
        w = fa_key_weights(qr, kc, lse, lens)
        kept, new = fa_cache_select(w, 500, lens, 4, 32)
        fa_cache_compact(kc, vc, kept, w)
        return a, b, qr, o, lse, kept, new, kc, vc, w

    want = [step(s) for s in sets]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[i] = step(sets[i])
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and fa_device_status() == 0
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("B,Hkv,Nk", [(1, 2, 8193), (3, 5, 12000), (2, 20, 9000), (8, 10, 8500)])
def test_select_clusters_of_every_size(B, Hkv, Nk):
    """Lists that one CTA could hold, shared by clusters of 8, 8, 2 and 1 (few lists, many lists)."""
    g = ref.gen(97 + Nk)
    w = torch.randint(0, 50, (B, Hkv, Nk), generator=g, device="cuda").float()   # many ties, across the cluster's parts
    lens = [max(1, Nk - 1000 * b) for b in range(B)]
    keep, first, recent = 1500, 7, 100
    kept, new = fa_cache_select(w, keep, ref.ints(lens), first, recent)
    assert new.tolist() == [min(n, keep) for n in lens]
    got, cpu = kept.tolist(), w.cpu()
    for b in range(B):
        for h in range(0, Hkv, max(1, Hkv // 3)):
            assert got[b][h] == ref.select(cpu[b, h], lens[b], keep, first, recent), (b, h)


def test_tensors_elsewhere_are_refused():
    g = ref.gen(98)
    q, k = ref.draw(g, 1, 2, 3, 64), ref.draw(g, 1, 2, 40, 64)
    par, lse = ref.ints([-1, 0, 1]), torch.zeros(1, 2, 3, device="cuda")
    for bad in (k.cpu(), None):
        with pytest.raises(TypeError):
            fa_fwd_tree(q, bad if bad is not None else par.tolist(), k, par)
        with pytest.raises(TypeError):
            fa_fwd_tree(q, k, bad, par)
    with pytest.raises(TypeError):
        fa_key_weights(q.cpu(), k, lse)
    with pytest.raises(ValueError):
        fa_fwd_tree(q, k, k, par.cpu())
    with pytest.raises(ValueError):
        fa_key_weights(q, k, lse.cpu())
    with pytest.raises(ValueError):
        fa_cache_compact(k, k.clone(), torch.zeros(1, 2, 4, dtype=torch.int32))


@pytest.mark.parametrize("Nq,d", [(1, 128), (33, 64), (700, 128), (700, 64)])
def test_weights_and_eviction_under_load(Nq, d):
    """Hundreds of launches back to back, copies running beside them: every one finishes in time with the same bits."""
    g = ref.gen(99)
    B, H, Hkv, Nk, keep = 3, 8, 4, 5000, 1000
    q, k = ref.draw(g, B, H, Nq, d), ref.draw(g, B, Hkv, Nk, d)
    lens = ref.ints([5000, 4097, 900])
    lse = torch.rand(B, H, Nq, generator=g, device="cuda") + 8
    want = fa_key_weights(q, k, lse, lens, True)
    rows, new = fa_cache_select(want, keep, lens, 4, 64)
    a, b = torch.empty(1 << 27, device="cuda", dtype=torch.uint8), torch.empty(1 << 27, device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    for _ in range(6):
        with torch.cuda.stream(side):
            for _ in range(8):
                a.copy_(b)
        outs = []
        for _ in range(32):
            w = fa_key_weights(q, k, lse, lens, True)
            outs.append((w, *fa_cache_select(w, keep, lens, 4, 64)))
        torch.cuda.synchronize()
        assert fa_device_status() == 0
        for w, r, n in outs:
            assert torch.equal(w, want) and torch.equal(r, rows) and torch.equal(n, new)
