"""The cache operators together, as a serving loop makes the calls: a prompt
rotated and attended to, its keys weighed, the cache cut back, a drafted tree
rotated into the cache and verified, its accepted branch made the next rows,
one more token decoded.  Beside it a plain 64-bit program keeps its own cache
and does every step by its definition; each step starts from the same bf16
cache rows, so the bounds are those of the single calls.

Bounds.  Rotated rows: half a bf16 step, 2^-8, of the result and fp32 angles
(2^-20 of the pair).  O: check_o of parity.py.  lse: 1e-4.  Weights: relative
1e-4 of the sum plus 1e-6, from the lse's 1e-4 in every term.
"""
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import (fa_cache_compact, fa_cache_select, fa_device_status, fa_fwd_decode, fa_fwd_strided,
                                      fa_fwd_tree, fa_key_weights, fa_rope, fa_rope_append, fa_rope_bwd,
                                      fa_rope_frequencies, fa_bwd)
from parity import check_o

pytestmark = pytest.mark.gpu


def near_rope(got, x, pos, freq, what):
    y, mag = ref.rope(x, pos, freq, 2 * freq.numel(), False, 1.0)
    err = (got.double() - y).abs()
    assert bool((err <= 2.0 ** -8 * y.abs() + 2.0 ** -20 * mag + 1e-30).all()), f"{what}: {float(err.max()):.3e}"


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_evict_draft_accept_decode(d):
    g = ref.gen(200 + d)
    B, H, Hkv, N, Nk, Nt = 2, 4, 2, 500, 700, 12
    G, scale = H // Hkv, 1 / math.sqrt(d)
    freq, _ = fa_rope_frequencies(d, scaling="base", factor=4.0)
    kc = torch.full((B, Nk, Hkv, d), math.nan, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    vc = torch.full((B, Nk, Hkv, d), math.nan, device="cuda", dtype=torch.bfloat16).transpose(1, 2)

    # ---- the prompt: rotate, store, attend, weigh
    q, k, v = ref.draw(g, B, H, N, d), ref.draw(g, B, Hkv, N, d), ref.draw(g, B, Hkv, N, d)
    lens = ref.ints([N] * B)
    qr = fa_rope_append(q, k, v, kc, vc, lens, freq)
    pos = torch.arange(N, device="cuda").expand(B, N)
    near_rope(qr, q, pos, freq, "q of the prompt")
    near_rope(kc[:, :, :N], k, pos, freq, "k of the prompt")
    assert torch.equal(vc[:, :, :N], v) and bool(torch.isnan(kc[:, :, N:]).all())
    share = lambda t: t[:, :, :N].repeat_interleave(G, 1)  # noqa: E731
    o, lse = fa_fwd_strided(qr, share(kc), share(vc), True)
    w = fa_key_weights(qr, kc, lse, lens, True)
    tri = torch.ones(N, N, dtype=torch.bool).tril().cuda()
    for b in range(B):
        for hk in range(Hkv):
            heads = slice(hk * G, hk * G + G)
            want = ref.key_weights(qr[b, heads], kc[b, hk], lse[b, heads], N, True, scale)
            assert bool(((w[b, hk].double() - want).abs() <= 1e-4 * want + 1e-6).all())
        wo, _, spread = ref.attention(qr[b, 0], kc[b, 0, :N], vc[b, 0, :N], tri, scale)
        check_o(o[b, 0], wo, f"prompt b{b}", spread)
    assert bool((w[:, :, N:] == 0).all())

    # ---- the cache cut back to 300 rows, in place
    keep, first, recent = 300, 4, 64
    kept, lens = fa_cache_select(w, keep, lens, first, recent)
    rows = [[ref.select(w[b, h].cpu(), N, keep, first, recent) for h in range(Hkv)] for b in range(B)]
    assert kept.tolist() == rows and lens.tolist() == [keep] * B
    k0, v0, w0 = kc.clone(), vc.clone(), w.clone()
    fa_cache_compact(kc, vc, kept, w)
    for b in range(B):
        for h in range(Hkv):
            at = torch.tensor(rows[b][h], device="cuda")
            assert torch.equal(kc[b, h, :keep], k0[b, h, at]) and torch.equal(vc[b, h, :keep], v0[b, h, at])
            assert torch.equal(w[b, h, :keep], w0[b, h, at])

    # ---- a drafted tree: rotated by its own positions into the cache, verified
    par = [[-1, 0, 0, 1, 1, 2, 3, -1, 7, 8, 8, 10], [-1, 0, 1, 2, 3, 4, 4, 5, -2, -2, -2, -2]]
    depth = [[0] * Nt for _ in range(B)]
    for b in range(B):
        for i, p in enumerate(par[b]):
            depth[b][i] = depth[b][p] + 1 if p >= 0 else 0
    parents, tree_pos = ref.ints(par), ref.ints(depth) + N  # positions go on behind the prompt's
    lens = lens + Nt
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nt, d), ref.draw(g, B, Hkv, Nt, d)
    k[1, :, 8:], v[1, :, 8:] = math.nan, math.inf           # padding nodes carry anything
    qr = fa_rope_append(q, k, v, kc, vc, lens, freq, tree_pos)
    near_rope(qr, q, tree_pos, freq, "q of the tree")
    near_rope(kc[0, :, keep:keep + Nt][None], k[:1], tree_pos[:1], freq, "k of the tree")
    o, lse = fa_fwd_tree(qr, kc, vc, parents, lens)
    for b in range(B):
        mask = ref.tree_mask(par[b], keep + Nt, Nt, Nk).cuda()
        live = mask.any(1)
        assert int(live.sum()) == (12, 8)[b]
        for h in range(H):
            wo, wl, spread = ref.attention(qr[b, h], kc[b, h // G], vc[b, h // G], mask, scale)
            check_o(o[b, h][live], wo[live], f"tree b{b} h{h}", spread[live])
            assert float((lse[b, h][live].double() - wl[live]).abs().max()) <= 1e-4
            assert bool((lse[b, h][~live] == -math.inf).all()) and bool((o[b, h][~live] == 0).all())

    # ---- the accepted branches become the next rows, and are weighed
    accepted = ref.ints([[0, 1, 4, -1], [0, 1, 2, 3]])
    k0 = kc.clone()
    fa_cache_compact(kc, vc, accepted, base=lens - Nt)
    for b, nodes in enumerate([[0, 1, 4], [0, 1, 2, 3]]):
        assert torch.equal(kc[b, :, keep:keep + len(nodes)], k0[b, :, [keep + x for x in nodes]])
    lens = ref.ints([keep + 3, keep + 4])
    m = 4  # the branches' queries, last rows of their sequences; the shorter one padded in front
    qa = torch.stack([torch.cat([q.new_zeros(H, 1, d), qr[0, :, [0, 1, 4]]], 1), qr[1, :, [0, 1, 2, 3]]])
    la = torch.stack([torch.cat([lse.new_full((H, 1), -math.inf), lse[0, :, [0, 1, 4]]], 1), lse[1, :, [0, 1, 2, 3]]])
    before = w.clone()
    fa_key_weights(qa, kc, la, lens, True, weights_in=w, weights=w)
    for b in range(B):
        n = int(lens[b])
        for hk in range(Hkv):
            heads = slice(hk * G, hk * G + G)
            add = ref.key_weights(qa[b, heads], kc[b, hk], la[b, heads], n, True, scale)
            want = before[b, hk].double() + add
            assert bool(((w[b, hk].double() - want).abs() <= 1e-4 * add + 2.0 ** -23 * want + 1e-6).all())
            # each query row spreads a weight of one over the rows it sees
            assert abs(float(add.sum()) - G * (n - keep)) <= 1e-3 * G * m

    # ---- one more token: the tree call with a single node is the decode call with shared heads
    lens = lens + 1
    q, k, v = ref.draw(g, B, H, 1, d), ref.draw(g, B, Hkv, 1, d), ref.draw(g, B, Hkv, 1, d)
    one = ref.ints([[N + 3], [N + 4]])
    qr = fa_rope_append(q, k, v, kc, vc, lens, freq, one, q_out=q)
    o, lse = fa_fwd_tree(qr, kc, vc, ref.ints([-1]), lens)
    od, ld = fa_fwd_decode(qr, kc.repeat_interleave(G, 1), vc.repeat_interleave(G, 1), lens, False)
    assert float((lse - ld).abs().max()) <= 2e-4
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            wo, wl, spread = ref.attention(qr[b, h], kc[b, h // G, :n], vc[b, h // G, :n],
                                           torch.ones(1, n, dtype=torch.bool, device="cuda"), scale)
            check_o(o[b, h], wo, f"decode b{b} h{h}", spread)
    assert fa_device_status() == 0


def test_training_step_through_rotation():
    """Rotation, attention and both backward passes: the gradients of q and k against the 64-bit program's.
    dq, dk within 2e-2 of the largest gradient, the bound of fa_bwd, whose result fa_rope_bwd turns and rounds once
    more (2^-8 of itself)."""
    from exact_attention_48_gb300 import fa_fwd

    g = ref.gen(210)
    B, H, N, d = 1, 2, 200, 64
    freq, _ = fa_rope_frequencies(32)
    q, k, v, do = (ref.draw(g, B, H, N, d) for _ in range(4))
    qr, kr = fa_rope(q, k, freq, interleaved=True)
    o, lse = fa_fwd(qr, kr, v, True)
    dqr, dkr, dv = fa_bwd(qr, kr, v, o, do, lse, True)
    dq, dk = fa_rope_bwd(dqr, dkr, freq, interleaved=True)
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    pos = torch.arange(N, device="cuda").expand(B, N)
    a, b = (ref_rope(t, pos, freq) for t in leaves[:2])
    s = (a @ b.transpose(-1, -2) / math.sqrt(d)).masked_fill(
        ~torch.ones(N, N, dtype=torch.bool, device="cuda").tril(), -math.inf)
    (torch.softmax(s, -1) @ leaves[2]).backward(do.double())
    for name, got, leaf in (("dq", dq, leaves[0]), ("dk", dk, leaves[1]), ("dv", dv, leaves[2])):
        want = leaf.grad
        bound = 2e-2 * float(want.abs().max()) + 2.0 ** -8 * want.abs()
        assert bool(((got.double() - want).abs() <= bound).all()), name
    assert fa_device_status() == 0


def ref_rope(x, pos, freq):
    """The interleaved rotation, differentiable."""
    rot = 2 * freq.numel()
    a = pos.double()[:, None, :, None] * freq.double()
    x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack((x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)
