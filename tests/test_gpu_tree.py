"""Attention of drafted trees over a cache (fa_fwd_tree) against 64 bits.

Bounds as for the other calls whose weights are rounded to bf16 before the
P V product (see parity.py): O within the flat 1e-2 or half a bf16 step plus
2^-8 of the spread; lse within 1e-4 (fp32 scores of 64 or 128 products).
"""
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import FaError, fa_device_status, fa_fwd_decode, fa_fwd_tree, fa_tree_workspace_bytes
from parity import check_o

pytestmark = pytest.mark.gpu


def trees(g, B, Nt):
    """Random trees; in every second one the last nodes are padding and one node has a bad parent."""
    u = torch.rand(B, Nt, generator=g, device="cuda")
    i = torch.arange(Nt, device="cuda")
    par = (u * (i + 1)).floor().clamp(max=Nt - 1).long()
    par = (torch.minimum(par, i) - 1).to(torch.int32)
    for b in range(1, B, 2):
        par[b, Nt - Nt // 4:] = -2
        par[b, Nt // 2] = Nt // 2 if b % 4 == 1 else 10 ** 6
    return par


def check(q, k, v, par, lens, o, lse, scale, what):
    B, H, Nt, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    rows = par.tolist() if par.dim() == 2 else [par.tolist()] * B
    for b in range(B):
        mask = ref.tree_mask(rows[b], lens[b], Nt, Nk).cuda()
        live = mask.any(1)
        for h in range(H):
            hk = h // (H // Hkv)
            want, wl, spread = ref.attention(q[b, h], k[b, hk], v[b, hk], mask, scale)
            tag = f"{what} b{b} h{h}"
            assert bool((o[b, h][~live] == 0).all()) and bool((lse[b, h][~live] == -math.inf).all()), f"{tag}: padding"
            if bool(live.any()):
                check_o(o[b, h][live], want[live], tag, spread[live])
                err = (lse[b, h][live].double() - wl[live]).abs().max()
                assert float(err) <= 1e-4, f"{tag}: lse {float(err):.3e}"


@pytest.mark.parametrize("B,H,Hkv,Nt,Nk,d,layout", [
    (1, 1, 1, 1, 1, 64, "bhnd"),
    (2, 2, 2, 1, 130, 128, "bhnd"),
    (4, 4, 2, 5, 300, 128, "bhnd"),
    (5, 8, 1, 33, 700, 64, "bnhd"),
    (4, 4, 4, 64, 513, 128, "pitch"),
    (2, 8, 2, 128, 1500, 128, "bnhd"),
    (2, 16, 1, 17, 260, 128, "bhnd"),
    (2, 2, 1, 128, 128, 64, "bhnd"),
    (1, 20, 1, 100, 901, 64, "bhnd"),
    (1, 2, 2, 65, 20001, 128, "bhnd"),
    (3, 6, 2, 12, 5003, 64, "bnhd"),
    (40, 2, 1, 3, 300, 64, "bhnd"),
    (37, 4, 2, 4, 1700, 64, "bhnd"),
    (400, 1, 1, 2, 140, 64, "bhnd"),
])
def test_tree(B, H, Hkv, Nt, Nk, d, layout):
    g = ref.gen(Nt + Nk)
    q = ref.draw(g, B, H, Nt, d, "bnhd" if layout == "bnhd" else "bhnd")
    k, v = ref.draw(g, B, Hkv, Nk, d, layout), ref.draw(g, B, Hkv, Nk, d, layout)
    par = trees(g, B, Nt)
    lens = ([Nk, Nk - Nk // 3, Nt, Nt // 2, 0] * B)[:B]
    o, lse = fa_fwd_tree(q, k, v, par, ref.ints(lens))
    assert fa_device_status() == 0
    check(q, k, v, par, lens, o, lse, 1 / math.sqrt(d), f"Nt{Nt} Nk{Nk}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales_and_shared_tree(d, scale):
    g = ref.gen(40 + d)
    B, H, Hkv, Nt, Nk = 2, 4, 2, 40, 401
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    par = trees(g, 1, Nt)[0]
    o, lse = fa_fwd_tree(q, k, v, par, None, scale)
    assert fa_device_status() == 0
    check(q, k, v, par, [Nk] * B, o, lse, scale, f"scale {scale}")


@pytest.mark.parametrize("d", [64, 128])
def test_hidden_rows_hold_anything(d):
    """Infinities and NaN behind a sequence's end and in padding nodes' rows reach nothing."""
    g = ref.gen(50)
    B, H, Hkv, Nt, Nk = 4, 4, 2, 24, 300
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    par = trees(g, B, Nt)
    lens = [300, 250, 24, 131]
    for b, n in enumerate(lens):
        used = ref.tree_mask(par[b].tolist(), n, Nt, Nk).any(0).cuda()
        for t, bad in ((k, math.nan), (v, math.inf), (v, math.nan)):
            t[b, :, ~used] = bad
        v[b, 1, ~used] = -math.inf
    o, lse = fa_fwd_tree(q, k, v, par, ref.ints(lens))
    assert fa_device_status() == 0 and bool(torch.isfinite(o).all())
    check(q, k, v, par, lens, o, lse, 1 / math.sqrt(d), "hidden")


def test_bad_lengths_are_clamped():
    g = ref.gen(51)
    q, k, v = ref.draw(g, 3, 2, 6, 128), ref.draw(g, 3, 2, 200, 128), ref.draw(g, 3, 2, 200, 128)
    par = trees(g, 3, 6)
    o, lse = fa_fwd_tree(q, k, v, par, ref.ints([-7, 10 ** 6, 199]))
    assert fa_device_status() == 0
    check(q, k, v, par, [0, 200, 199], o, lse, 1 / math.sqrt(128), "clamped")


@pytest.mark.parametrize("d", [64, 128])
def test_a_chain_is_the_causal_decode(d):
    g = ref.gen(52)
    B, H, Nt, Nk = 2, 3, 6, 1000
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, H, Nk, d), ref.draw(g, B, H, Nk, d)
    cl = ref.ints([1000, 717])
    o, lse = fa_fwd_tree(q, k, v, ref.ints(list(range(-1, Nt - 1))), cl)
    od, ld = fa_fwd_decode(q, k, v, cl, True)
    assert float((lse - ld).abs().max()) <= 2e-4       # each within 1e-4 of the exact one
    # O: half a bf16 step each, and 2^-8 of the spread (|v - o| below 6 here) for each side's rounded weights
    assert float((o.float() - od.float()).abs().max()) <= 2e-2


def test_sharp_scores():
    """Scores in the hundreds: one key carries the row, and maxima move from tile to tile."""
    g = ref.gen(53)
    B, H, Hkv, Nt, Nk, d = 1, 4, 2, 31, 2000, 128
    q, k, v = ref.draw(g, B, H, Nt, d, mult=4.0), ref.draw(g, B, Hkv, Nk, d, mult=4.0), ref.draw(g, B, Hkv, Nk, d)
    k *= torch.linspace(0.5, 1.5, Nk, device="cuda").to(torch.bfloat16)[:, None]
    par = trees(g, B, Nt)
    o, lse = fa_fwd_tree(q, k, v, par)
    mask = ref.tree_mask(par[0].tolist(), Nk, Nt, Nk).cuda()
    for h in range(H):
        want, wl, spread = ref.attention(q[0, h], k[0, h // 2], v[0, h // 2], mask, 1 / math.sqrt(d))
        check_o(o[0, h], want, "sharp", spread)
        # scores up to ~600: fp32 rounds them to 2^-24 * 600 * a few operations
        assert float((lse[0, h].double() - wl).abs().max()) <= 1e-3


def test_long_cache_offsets_past_2_31():
    g = ref.gen(54)
    H, Nt, Nk, d = 2, 3, (1 << 24) + 77, 128
    q = ref.draw(g, 1, H, Nt, d)
    k = torch.empty(1, 1, Nk, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    v = torch.empty(1, 1, Nk, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    assert k.numel() > 1 << 31
    v[0, 0, -100:] += 1.0
    k[0, 0, -50] = q[0, 0, 0] * 3          # a key that node 0 of head 0 attends to strongly
    par = ref.ints([-1, 0, -1])
    o, lse = fa_fwd_tree(q, k, v, par)
    assert fa_device_status() == 0
    scale = 1 / math.sqrt(d)
    for h in range(H):
        for i in range(Nt):
            hide = [j for j in range(i) if not (i == 1 and j == 0)] + list(range(i + 1, Nt))
            parts, outs = [], []
            for j0 in range(0, Nk, 1 << 21):
                kk, vv = k[0, 0, j0:j0 + (1 << 21)].double(), v[0, 0, j0:j0 + (1 << 21)].double()
                t = kk @ q[0, h, i].double() * scale
                for x in hide:
                    if 0 <= Nk - Nt + x - j0 < t.numel():
                        t[Nk - Nt + x - j0] = -math.inf
                parts.append(torch.logsumexp(t, 0))
                outs.append(torch.softmax(t, 0) @ vv)
            ls = torch.stack(parts)
            wl = torch.logsumexp(ls, 0)
            want = ((ls - wl).exp()[:, None] * torch.stack(outs)).sum(0)
            assert abs(float(lse[0, h, i]) - float(wl)) <= 1e-4
            assert float((o[0, h, i].double() - want).abs().max()) <= 1e-2


@pytest.mark.parametrize("H,Hkv,Nt,Nk,d", [(16, 8, 64, 9000, 64), (8, 8, 1, 9000, 64), (16, 8, 64, 9000, 128),
                                           (32, 8, 64, 5000, 64), (32, 8, 64, 5000, 128)])
def test_many_launches_under_load(H, Hkv, Nt, Nk, d):
    """Hundreds of launches back to back, other copies running beside them: every one finishes in time and gives
    the same bits (the softmax, product and load roles may overtake each other as far as their barriers let them)."""
    g = ref.gen(58)
    B = 4
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    par, cl = trees(g, B, Nt), ref.ints([Nk, Nk - 5, Nk // 2, 3 * Nk // 4])
    want, wl = fa_fwd_tree(q, k, v, par, cl)
    a, b = torch.empty(1 << 27, device="cuda", dtype=torch.uint8), torch.empty(1 << 27, device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    for _ in range(8):
        with torch.cuda.stream(side):
            for _ in range(8):
                a.copy_(b)
        outs = [fa_fwd_tree(q, k, v, par, cl) for _ in range(32)]
        torch.cuda.synchronize()
        assert fa_device_status() == 0
        for o, lse in outs:
            assert torch.equal(o, want) and torch.equal(lse, wl)


def test_outputs_only_and_workspace():
    """o in a wider buffer, lse between guards, a caller's workspace: nothing else is written; runs repeat bitwise."""
    g = ref.gen(55)
    B, H, Hkv, Nt, Nk, d = 3, 8, 2, 9, 3001, 128
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    par, cl = trees(g, B, Nt), ref.ints([3001, 1500, 4])
    want, wl = fa_fwd_tree(q, k, v, par, cl)
    buf = torch.full((B, Nt + 2, H, d + 16), 7.0, device="cuda", dtype=torch.bfloat16)
    o = buf[:, 1:1 + Nt, :, 8:8 + d].transpose(1, 2)
    lbuf = torch.full((B * H * Nt + 8,), 7.0, device="cuda")
    lse = lbuf[4:4 + B * H * Nt].view(B, H, Nt)
    need = fa_tree_workspace_bytes(B, H, Hkv, Nt, Nk, d)
    ws = torch.full((need + 512,), 99, device="cuda", dtype=torch.uint8)
    for _ in range(2):
        fa_fwd_tree(q, k, v, par, cl, o=o, lse=lse, workspace=ws[:need] if need else None)
        assert torch.equal(o, want) and torch.equal(lse, wl)
        buf2 = buf.clone()
        buf2[:, 1:1 + Nt, :, 8:8 + d] = 7.0
        assert bool((buf2 == 7.0).all()) and bool((lbuf[:4] == 7.0).all()) and bool((lbuf[-4:] == 7.0).all())
        assert bool((ws[need:] == 99).all())
    if need:
        with pytest.raises(FaError):
            fa_fwd_tree(q, k, v, par, cl, workspace=ws[:need - 1])


def test_streams_and_two_captured_graphs():
    """Two graphs captured with the library's own workspace and replayed in turn; a call on another stream."""
    g = ref.gen(56)
    B, H, Hkv, Nt, Nk, d = 2, 4, 2, 16, 2500, 64
    sets = []
    for _ in range(2):
        q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
        par, cl = trees(g, B, Nt), ref.ints([2500, 1234])
        o, lse = torch.empty_like(q), torch.empty(B, H, Nt, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa_fwd_tree(q, k, v, par, cl, o=o, lse=lse)
        sets.append((q, k, v, par, cl, o, lse, graph))
    sets[0][4].copy_(ref.ints([100, 2499]))   # lengths are read at replay
    sets[0][7].replay()
    sets[1][7].replay()
    sets[0][7].replay()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for q, k, v, par, cl, o, lse, _ in sets:
        s.wait_stream(torch.cuda.current_stream())
        a, b = fa_fwd_tree(q, k, v, par, cl, stream=s)
        s.synchronize()
        assert torch.equal(a, o) and torch.equal(b, lse)
    assert fa_device_status() == 0


def test_refusals():
    q = torch.zeros(1, 4, 8, 64, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(1, 2, 32, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    par = ref.ints([-1] * 8)
    with pytest.raises(ValueError):
        fa_fwd_tree(q[:, :3], k, v, par)                                  # 3 heads over 2
    with pytest.raises(ValueError):
        fa_fwd_tree(q, k, v[:, :, :31], par)
    with pytest.raises(ValueError):
        fa_fwd_tree(q, k, v, par.long())
    with pytest.raises(ValueError):
        fa_fwd_tree(q, k, v, par[:7])
    with pytest.raises(ValueError):
        fa_fwd_tree(q, k, v, par, ref.ints([1, 2]))
    with pytest.raises(FaError):
        fa_fwd_tree(q, k, v, par, scale=math.nan)
    with pytest.raises(FaError):
        fa_fwd_tree(q, k, v, par, o=q)
    with pytest.raises(FaError):
        fa_fwd_tree(q.repeat(1, 1, 17, 1), k, v, ref.ints([-1] * 136))    # more than 128 nodes
    with pytest.raises(TypeError):
        fa_fwd_tree(q.half(), k, v, par)


def test_workspace_taken_by_the_library():
    """The C call with a null workspace takes it on the stream; two captured graphs of it do not share it."""
    import ctypes

    from exact_attention_48_gb300 import fa_key_weights
    from exact_attention_48_gb300.binding import library
    g = ref.gen(57)
    B, H, Hkv, Nt, Nk, d = 2, 4, 2, 9, 2000, 128
    lib = library()
    st = lambda t: (ctypes.c_int64 * 3)(*t.stride()[:3])  # noqa: E731
    sets = []
    for _ in range(2):
        q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
        par = trees(g, B, Nt)
        o, lse = torch.empty_like(q), torch.empty(B, H, Nt, device="cuda")

        def call():
            return lib.fa_fwd_tree(q.data_ptr(), st(q), k.data_ptr(), st(k), v.data_ptr(), st(v), o.data_ptr(), st(o),
                                   lse.data_ptr(), par.data_ptr(), Nt, None, B, H, Hkv, Nt, Nk, d, 1 / math.sqrt(d),
                                   None, 0, torch.cuda.current_stream().cuda_stream)
        assert call() == 0
        want = fa_fwd_tree(q, k, v, par)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            assert call() == 0
        sets.append((o, lse, want, graph, (q, k, v, par)))  # a graph does not keep its inputs alive
    for o, lse, *_ in sets:
        o.zero_(), lse.zero_()
    for i in (0, 1, 1, 0):
        sets[i][3].replay()
    torch.cuda.synchronize()
    for o, lse, want, *_ in sets:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # the key weights' partial sums likewise
    q, k = ref.draw(g, 1, 2, 700, d), ref.draw(g, 1, 1, 600, d)
    lse = torch.full((1, 2, 700), 6.0, device="cuda")
    assert lib.fa_key_weights_workspace_bytes(1, 2, 1, 700, 600, d) > 0
    w = torch.empty(1, 1, 600, device="cuda")
    rc = lib.fa_key_weights(q.data_ptr(), st(q), k.data_ptr(), st(k), lse.data_ptr(), None, w.data_ptr(), None, 1, 2, 1,
                            700, 600, d, 1, 0.1, None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(w, fa_key_weights(q, k, lse, None, True, 0.1))
