"""Drafted-tree attention where scores are not finite: a NaN that a node sees
reaches that node's results and no other row's, a score of -inf weighs
nothing, and neither is lost between the runs that a long cache is cut into.
Rows whose 64-bit result is finite keep the bounds of test_gpu_tree.py."""
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import fa_device_status, fa_fwd_tree
from parity import check_o

pytestmark = pytest.mark.gpu

# one row tile and two; a cache in one run a unit and cut into several; more sequences than a warp
SHAPES = [(2, 4, 2, 8, 300), (2, 4, 2, 8, 5000), (2, 8, 2, 48, 200), (2, 8, 2, 48, 3001), (40, 2, 1, 3, 1500)]


def forest(B, Nt):
    """Two branches from every root, the last node of odd sequences padding."""
    par = torch.tensor([[(i - 1) // 2 if i else -1 for i in range(Nt)]] * B, dtype=torch.int32)
    par[1::2, Nt - 1] = -2
    return par.cuda()


def compare(q, k, v, par, lens, scale, what):
    """Returns how many live rows came out as NaN."""
    B, H, Nt, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    o, lse = fa_fwd_tree(q, k, v, par, ref.ints(lens), scale)
    assert fa_device_status() == 0
    bad = 0
    for b in range(B):
        mask = ref.tree_mask(par[b].tolist(), lens[b], Nt, Nk).cuda()
        live = mask.any(1)
        for h in range(H):
            hk = h * Hkv // H
            want, wl, spread = ref.attention(q[b, h], k[b, hk], v[b, hk], mask, scale)
            tag = f"{what} b{b} h{h}"
            assert bool((o[b, h][~live] == 0).all()) and bool((lse[b, h][~live] == -math.inf).all()), f"{tag}: padding"
            none = live & (wl == -math.inf)          # scores of -inf alone: as a row that sees nothing
            assert bool((o[b, h][none] == 0).all()) and bool((lse[b, h][none] == -math.inf).all()), f"{tag}: no weight"
            fine = live & torch.isfinite(wl) & torch.isfinite(want).all(1)
            nan = live & ~fine & ~none
            lost = nan & ~(torch.isnan(o[b, h]).all(1) & ~torch.isfinite(lse[b, h]))
            assert not bool(lost.any()), f"{tag}: rows {lost.nonzero()[:, 0].tolist()} hide a NaN"
            bad += int(nan.sum())
            if bool(fine.any()):
                check_o(o[b, h][fine], want[fine], tag, spread[fine])
                assert float((lse[b, h][fine].double() - wl[fine]).abs().max()) <= 1e-4, tag
    return bad


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,Nt,Nk", SHAPES)
def test_nan_in_a_query_row(B, H, Hkv, Nt, Nk, d):
    g = ref.gen(400 + Nk)
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    q[0, 1, Nt // 2, 3] = math.nan
    q[1, 0, 0] = math.nan
    q[1, 0, Nt - 1] = math.nan                      # padding
    assert compare(q, k, v, forest(B, Nt), [Nk - 77 * (b % 2) for b in range(B)], d ** -0.5, "query") == 2


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,Nt,Nk", SHAPES)
def test_nan_in_key_rows(B, H, Hkv, Nt, Nk, d):
    """Before the tree (every row of the cache head sees it) and in a node's row (its branch sees it)."""
    g = ref.gen(401 + Nk)
    lens = [Nk - 77 * (b % 2) for b in range(B)]
    for place in ("first rows", "last rows before the tree", "a node"):
        q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
        row = {"first rows": 5, "last rows before the tree": lens[0] - Nt - 1, "a node": lens[0] - Nt + 1}[place]
        k[0, Hkv - 1, row] = math.nan
        bad = compare(q, k, v, forest(B, Nt), lens, d ** -0.5, place)
        assert bad > 0 if place == "a node" else bad == H // Hkv * Nt


@pytest.mark.parametrize("scale", [0.1, -0.1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,Nt,Nk", SHAPES)
def test_infinite_scores(B, H, Hkv, Nt, Nk, d, scale):
    """Infinite key elements: scores of -inf or +inf by the sign of the query element.  Rows that meet -inf alone go
    on as if the keys were not there, though a whole tile, run or sequence of them comes first."""
    g = ref.gen(402 + Nk)
    lens = [Nk - 77 * (b % 2) for b in range(B)]
    for n in (1, 150, 1100, Nk):
        q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
        k[..., 7] = 0.0
        k[0, 0, :n, 7] = -math.inf if scale > 0 else math.inf
        q[..., 7] = q[..., 7].abs() + 0.5
        q[0, 0, 0, 7] = -1.0
        compare(q, k, v, forest(B, Nt), lens, scale, f"{n} rows")
