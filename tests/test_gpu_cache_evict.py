"""Eviction (fa_cache_select, fa_cache_compact): whole numbers and copies, so
every comparison is exact."""
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import FaError, fa_cache_compact, fa_cache_select

pytestmark = pytest.mark.gpu


def check_select(w, lens, keep, first, recent):
    kept, new = fa_cache_select(w, keep, None if lens is None else ref.ints(lens), first, recent)
    B, Hkv, Nk = w.shape
    lens = [Nk] * B if lens is None else [max(0, min(n, Nk)) for n in lens]
    assert new.tolist() == [min(n, keep) for n in lens]
    got, cpu = kept.tolist(), w.cpu()
    for b in range(B):
        for h in range(Hkv):
            assert got[b][h] == ref.select(cpu[b, h], lens[b], keep, first, recent), (b, h)
    return kept, new


@pytest.mark.parametrize("B,Hkv,Nk,keep,first,recent", [
    (1, 1, 1, 1, 0, 0), (2, 3, 10, 4, 1, 1), (3, 2, 1000, 300, 4, 32), (2, 2, 4097, 1, 0, 0), (2, 1, 4097, 4097, 0, 0),
    (1, 2, 5000, 4999, 0, 1), (2, 2, 777, 100, 60, 40), (1, 3, 40000, 12345, 0, 1000), (2, 1, 33, 32, 0, 0),
    (1, 1, 300001, 1000, 16, 64)])
def test_select(B, Hkv, Nk, keep, first, recent):
    g = ref.gen(Nk + keep)
    w = torch.exp(2 * torch.randn(B, Hkv, Nk, generator=g, device="cuda"))
    check_select(w, None, keep, first, recent)
    check_select(w, [max(1, Nk - Nk // 3), keep, 0][:B], keep, first, recent)


@pytest.mark.parametrize("Nk", [65, 3000, 20000])
def test_select_ties_and_odd_values(Nk):
    """All alike, few values, both zeros, negatives, infinities, NaN, values that differ in the last bit."""
    g = ref.gen(80 + Nk)
    rows = [torch.zeros(Nk, device="cuda"), torch.full((Nk,), 0.25, device="cuda")]
    rows.append(torch.randint(0, 3, (Nk,), generator=g, device="cuda").float() - 1)
    z = torch.zeros(Nk, device="cuda")
    z[::2] = -0.0
    z[5] = 1e-45
    rows.append(z)
    odd = torch.randn(Nk, generator=g, device="cuda")
    odd[::7] = math.nan
    odd[1::11] = math.inf
    odd[2::13] = -math.inf
    rows.append(odd)
    step = 1.0 + torch.randint(0, 4, (Nk,), generator=g, device="cuda").float() * 2.0 ** -23
    rows.append(step)
    rows.append(torch.full((Nk,), math.nan, device="cuda"))
    rows.append(torch.arange(Nk, device="cuda").float())
    w = torch.stack(rows)[None]
    for keep in (1, Nk // 2, Nk - 1):
        check_select(w, None, keep, min(2, keep // 2), min(5, keep // 3))


def test_select_ignores_what_lies_behind():
    g = ref.gen(81)
    w = torch.rand(2, 2, 500, generator=g, device="cuda")
    w[0, :, 400:] = math.inf
    w[1, :, 33:] = math.nan
    check_select(w, [400, 33], 20, 3, 4)
    check_select(w, [10 ** 6, -4], 20, 3, 4)


def moved(x, y, kept, base, B, Hkv):
    """y with row base + i = x's row base + kept[i]."""
    y = y.clone()
    Nk, Nout = x.shape[2], y.shape[2]
    for b in range(B):
        for h in range(Hkv):
            rows = kept[b][h]
            s = [(base[b] + i, base[b] + r) for i, r in enumerate(rows)
                 if r >= 0 and 0 <= base[b] + i < Nout and 0 <= base[b] + r < Nk]
            if s:
                dst, src = (torch.tensor(z, device="cuda") for z in zip(*s))
                y[b, h, dst] = x[b, h, src]
    return y


@pytest.mark.parametrize("B,Hkv,Nk,keep,d,layout", [
    (1, 1, 1, 1, 64, "bhnd"), (2, 3, 300, 100, 128, "bhnd"), (1, 2, 5000, 2222, 64, "bnhd"),
    (2, 2, 1027, 1000, 128, "pitch"), (1, 1, 40000, 39999, 64, "bhnd"), (9, 4, 700, 333, 128, "bnhd")])
def test_evict_in_place_and_out(B, Hkv, Nk, keep, d, layout):
    g = ref.gen(82 + Nk)
    k, v = ref.draw(g, B, Hkv, Nk, d, layout), ref.draw(g, B, Hkv, Nk, d, layout)
    w = torch.rand(B, Hkv, Nk, generator=g, device="cuda")
    lens = ([Nk, keep // 2 + 1, Nk - Nk // 5] * B)[:B]
    kept, _ = check_select(w, lens, keep, min(3, keep // 3), keep // 4)
    rows, zero = kept.tolist(), [0] * B
    want = [moved(x, x, rows, zero, B, Hkv) for x in (k, v, w[..., None])]
    # out of place, into a buffer of its own with more rows than are moved
    ko, vo = (torch.full((B, Hkv, keep + 3, d), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    wo = torch.full((B, Hkv, keep + 3), 5.0, device="cuda")
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    fa_cache_compact(k, v, kept, w, None, ko, vo, wo)
    for x, y in ((k, ko), (v, vo), (w[..., None], wo[..., None])):
        assert torch.equal(y, moved(x, torch.full_like(y, 5.0), rows, zero, B, Hkv))
    assert torch.equal(k, k0) and torch.equal(v, v0) and torch.equal(w, w0)
    # any order out of place
    flip = kept.flip(-1).contiguous()
    ko.fill_(5.0), vo.fill_(5.0)
    fa_cache_compact(k, v, flip, k_out=ko, v_out=vo)
    assert torch.equal(ko, moved(k, torch.full_like(ko, 5.0), flip.tolist(), zero, B, Hkv))
    # in place
    out = fa_cache_compact(k, v, kept, w)
    assert out[0] is k and torch.equal(k, want[0]) and torch.equal(v, want[1]) and torch.equal(w, want[2][..., 0])


def test_in_place_every_row_moves_by_one():
    """The tightest order: every destination is the next row's source, over many chunks."""
    g = ref.gen(83)
    for d, Nk in ((128, 3001), (64, 10007)):
        k, v = ref.draw(g, 2, 2, Nk, d), ref.draw(g, 2, 2, Nk, d)
        w = torch.rand(2, 2, Nk, generator=g, device="cuda")
        k0, v0, w0 = k.clone(), v.clone(), w.clone()
        kept = torch.arange(1, Nk, dtype=torch.int32, device="cuda").expand(2, 2, Nk - 1).contiguous()
        fa_cache_compact(k, v, kept, w)
        assert torch.equal(k[:, :, :-1], k0[:, :, 1:]) and torch.equal(k[:, :, -1], k0[:, :, -1])
        assert torch.equal(v[:, :, :-1], v0[:, :, 1:]) and torch.equal(w[:, :, :-1], w0[:, :, 1:])


def test_accepted_branch():
    """base + shared lists: each sequence's accepted nodes become its next rows; rows off the end are skipped."""
    g = ref.gen(84)
    B, Hkv, Nk, d = 4, 2, 64, 128
    k, v = ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    kept = ref.ints([[0, 2, 5, 7], [1, -1, -1, -1], [0, 1, 2, 60], [3, 4, 9, -1]])
    base = [10, 55, 20, 61]
    k0, v0 = k.clone(), v.clone()
    rows = [[r] * Hkv for r in kept.tolist()]
    fa_cache_compact(k, v, kept, base=ref.ints(base))
    assert torch.equal(k, moved(k0, k0, rows, base, B, Hkv)) and torch.equal(v, moved(v0, v0, rows, base, B, Hkv))
    k, v = k0.clone(), v0.clone()
    far = [-2 ** 31, 2 ** 31 - 1, -3, 0]
    fa_cache_compact(k, v, kept, base=ref.ints(far))
    assert torch.equal(k, moved(k0, k0, rows, far, B, Hkv))


def test_bad_lists_touch_nothing_else():
    """Entries outside the cache are skipped; lists out of order in place give wrong rows inside [0, M) only."""
    g = ref.gen(85)
    k, v = ref.draw(g, 1, 1, 400, 64), ref.draw(g, 1, 1, 400, 64)
    k0 = k.clone()
    kept = torch.randint(-500, 900, (1, 1, 300), generator=g, device="cuda", dtype=torch.int32)
    kept[0, 0, 0] = 2 ** 31 - 1
    fa_cache_compact(k, v, kept)
    assert torch.equal(k[:, :, 300:], k0[:, :, 300:])
    skipped = ((kept < 0) | (kept >= 400))[0, 0].nonzero()[:, 0]
    assert torch.equal(k[0, 0, skipped], k0[0, 0, skipped])


def test_offsets_past_2_31():
    Nk, d = (1 << 23) + 100, 128
    k = torch.zeros(1, 2, Nk, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    assert k.numel() > 1 << 31
    k[0, 1, -5:] = torch.arange(1, 6, device="cuda", dtype=torch.bfloat16)[:, None]
    w = torch.zeros(1, 2, Nk, device="cuda")
    w[0, 1, -5:] = 1.0
    w[0, 0, 7] = 2.0
    kept, _ = fa_cache_select(w, 5)
    assert kept[0, 1].tolist() == list(range(Nk - 5, Nk)) and kept[0, 0].tolist() == [0, 1, 2, 3, 7]
    fa_cache_compact(k, v, kept, w)
    assert k[0, 1, :5, 0].tolist() == [1, 2, 3, 4, 5] and w[0, 1, :5].tolist() == [1] * 5


def test_streams_and_capture():
    g = ref.gen(86)
    B, Hkv, Nk, d, keep = 2, 2, 900, 64, 200
    k, v = ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    w = torch.rand(B, Hkv, Nk, generator=g, device="cuda")
    want = fa_cache_select(w, keep, first=4, recent=10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa_cache_select(w, keep, first=4, recent=10, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k1, v1, w1 = k.clone(), v.clone(), w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, _ = fa_cache_select(w1, keep, first=4, recent=10)
        fa_cache_compact(k1, v1, kept, w1)
    graph.replay()
    torch.cuda.synchronize()
    fa_cache_compact(k, v, want[0], w)
    assert torch.equal(k1, k) and torch.equal(v1, v) and torch.equal(w1, w)


def test_refusals():
    k, v = (torch.zeros(1, 2, 32, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.zeros(1, 2, 32, device="cuda")
    kept = torch.zeros(1, 2, 4, device="cuda", dtype=torch.int32)
    for keep in (0, 33):
        with pytest.raises(ValueError):
            fa_cache_select(w, keep)
    with pytest.raises(FaError):
        fa_cache_select(w, 8, first=5, recent=4)
    with pytest.raises(FaError):
        fa_cache_select(w, 8, first=-1)
    with pytest.raises(TypeError):
        fa_cache_select(w[0], 8)
    with pytest.raises(ValueError):
        fa_cache_compact(k, v, kept.long())
    with pytest.raises(ValueError):
        fa_cache_compact(k, v, kept, k_out=k)
    with pytest.raises(ValueError):
        fa_cache_compact(k, v, kept, w, None, k.clone(), v.clone())
    with pytest.raises(FaError):      # k in place, v not
        fa_cache_compact(k, v, kept, k_out=k, v_out=v.clone())
    with pytest.raises(FaError):      # swapped
        fa_cache_compact(k, v, kept, k_out=v, v_out=k)
