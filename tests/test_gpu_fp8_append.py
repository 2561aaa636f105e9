"""The append to a cache held in 8 bits (fa_rope_append_fp8) against its 64-bit
definition.

Bounds.  v takes no arithmetic before it is rounded: codes and scales are equal to
the last bit, and so are old rows that are rounded to a greater scale.  k is turned
in fp32, off by at most 2^-20 of |x1| + |x2| and the factor (as in test_gpu_rope.py):
its code is the nearest of some value within that of the exact one, so the value it
stands for is off by that and half a step of e4m3: 2^-4 of it, or 2^-10 of the
scale.  A scale of k may be the next power of two only where the greatest
value is that near to 448 times one.
"""
import math

import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import fa_rope, fa_rope_append_fp8, fa_rope_frequencies

pytestmark = pytest.mark.gpu


def check_k(got, got_scale, x, mag, n, codes, scale, block, factor, what):
    """One head of k: x [N, d] exact turned rows."""
    want, want_scale = r8.append(x, n, codes, scale, block)
    got, got_scale = got.double(), got_scale.double()
    N, Nk = x.shape[0], codes.shape[0]
    start = n - N
    off = 2.0 ** -20 * abs(factor) * mag
    for blk in range(scale.shape[0]):
        lo, hi = blk * block, min(Nk, (blk + 1) * block)
        new = range(max(lo, start, 0), min(hi, n))
        if not len(new):
            assert torch.equal(got[lo:hi].nan_to_num(777.0), codes[lo:hi].double().nan_to_num(777.0)), what
            assert float(got_scale[blk]) == float(scale[blk]) or scale[blk] != scale[blk], what
            continue
        s = float(got_scale[blk])
        if s != float(want_scale[blk]):
            a = float((x[[r - start for r in new]]).abs().max())
            lean = float(off.max())
            assert s in (r8.least_scale(a - lean), r8.least_scale(a + lean)), (what, blk, s, float(want_scale[blk]))
        y, near = x[[r - start for r in new]], off[[r - start for r in new]]
        err = (got[list(new)] * s - y).abs()
        assert bool((err <= near + torch.maximum(2.0 ** -4 * (y.abs() + near), torch.full_like(y, 2.0 ** -10 * s))).all()), \
            f"{what} block {blk}: {float(err.max()):.3e}"
        if lo < start:
            old = r8.round_e4m3(codes[lo:start].double() * (float(scale[blk]) / s))
            assert torch.equal(got[lo:start].nan_to_num(777.0), old.nan_to_num(777.0)), (what, blk, "old rows")
        if n < hi:
            assert torch.equal(got[max(n, lo):hi].nan_to_num(777.0), codes[max(n, lo):hi].double().nan_to_num(777.0)), what


def check_v(got, got_scale, x, n, codes, scale, block, what):
    want, want_scale = r8.append(x.double(), n, codes, scale, block)
    assert torch.equal(got_scale.double().nan_to_num(777.0), want_scale.nan_to_num(777.0)), what
    assert torch.equal(got.double().nan_to_num(777.0), want.nan_to_num(777.0)), what


def run(g, B, H, Hkv, N, Nk, d, rot, block, interleaved, layout, lens, factor=1.0, positions=None, mult=1.0, spread=6):
    q, k, v = (ref.draw(g, B, h, N, d, layout, mult) for h in (H, Hkv, Hkv))
    kc, ks = r8.cache(g, B, Hkv, Nk, d, block, layout, spread)
    vc, vs = r8.cache(g, B, Hkv, Nk, d, block, layout, spread)
    before = [t.clone() for t in (kc, ks, vc, vs)]
    freq, _ = fa_rope_frequencies(rot)
    lens_t = ref.ints(lens)
    qo = fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, lens_t, freq, positions, interleaved, factor, block)
    pos = lens_t[:, None] - N + torch.arange(N, device="cuda") if positions is None else positions.expand(B, N)
    y, mag = ref.rope(q, pos, freq, rot, interleaved, factor)
    assert bool(((qo.double() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -20 * abs(factor) * mag + 1e-30).all())
    x, mag = ref.rope(k, pos, freq, rot, interleaved, factor)
    for b in range(B):
        for h in range(Hkv):
            what = f"b{b} h{h}"
            check_k(kc[b, h], ks[b, h], x[b, h], mag[b, h], lens[b], before[0][b, h], before[1][b, h], block, factor, what)
            check_v(vc[b, h], vs[b, h], v[b, h], lens[b], before[2][b, h], before[3][b, h], block, what)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hkv,N,Nk,d,rot,block,layout", [
    (1, 1, 1, 1, 1, 64, 64, 64, "bhnd"),
    (3, 4, 2, 1, 300, 128, 128, 64, "bhnd"),
    (2, 8, 8, 1, 70, 64, 32, 128, "bnhd"),
    (2, 3, 1, 5, 100, 128, 48, 16, "pitch"),
    (4, 6, 2, 33, 257, 64, 16, 32, "bnhd"),
    (2, 4, 4, 130, 400, 128, 112, 128, "bhnd"),
    (1, 40, 5, 300, 301, 64, 64, 16, "bhnd"),
    (2, 2, 2, 257, 1000, 128, 64, 64, "pitch"),
    (5, 70, 10, 3, 64, 64, 64, 32, "bhnd"),
])
def test_append(B, H, Hkv, N, Nk, d, rot, block, layout, interleaved):
    g = ref.gen(1000 + N + Nk)
    lens = [N + (7 * b + 3 * Nk // 4) % (Nk - N + 1) for b in range(B)]
    run(g, B, H, Hkv, N, Nk, d, rot, block, interleaved, layout, lens)


def test_block_boundaries():
    """A single token at every place of a block, and runs that end at, before and behind its end."""
    g = ref.gen(1001)
    for n in (1, 15, 16, 17, 32, 33, 48):
        run(g, 2, 2, 2, 1, 48, 64, 64, 16, False, "bhnd", [n, max(1, n - 1)])
    for N in (15, 16, 17, 31, 32, 33):
        run(g, 2, 1, 1, N, 64, 64, 64, 16, False, "bhnd", [N, 64])
        run(g, 2, 1, 1, N, 64, 64, 64, 16, False, "bhnd", [N + 1, N + 15])


def test_rows_outside_the_cache():
    """cache_seqlens is not clamped: rows before 0 or behind Nk are not written, q is turned all the same."""
    g = ref.gen(1002)
    run(g, 6, 2, 2, 40, 100, 64, 64, 32, False, "bhnd", [10, 39, 40, 110, 139, 100])
    run(g, 4, 2, 1, 5, 20, 128, 128, 16, True, "bnhd", [0, -3, 25, 1000])


def test_scale_grows_and_codes_follow():
    """The new row is greater than the block's: the rows before it are rounded to the new scale, tiny ones away."""
    g = ref.gen(1003)
    for mult in (1e-6, 1.0, 1e4, 1e30):
        run(g, 2, 2, 2, 1, 64, 64, 64, 64, False, "bhnd", [20, 64], mult=mult, spread=9)


def test_scale_of_an_empty_block_is_not_read():
    g = ref.gen(1004)
    q, k, v = (ref.draw(g, 1, 1, 2, 64) for _ in range(3))
    kc, ks = r8.cache(g, 1, 1, 64, 64, 16)
    ks.fill_(math.nan)
    ks[..., 0] = 1.0
    vc, vs = kc.clone(), ks.clone()
    freq, _ = fa_rope_frequencies(64)
    fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, ref.ints([18]), freq, block=16)
    assert float(vs[0, 0, 1]) == r8.least_scale(float(v.abs().max())) and math.isfinite(float(ks[0, 0, 1]))
    assert float(ks[0, 0, 0]) == 1.0 and bool(torch.isnan(ks[0, 0, 2:]).all())


def test_zeros_infinities_and_nan():
    """A block of zeros takes the least scale; what is not finite becomes NaN and does not count for the scale."""
    v = torch.zeros(1, 1, 3, 64, device="cuda", dtype=torch.bfloat16)
    q = k = torch.zeros_like(v)
    codes = torch.zeros(1, 1, 16, 64, device="cuda").to(r8.E4M3)
    freq, _ = fa_rope_frequencies(64)

    def one(v):
        kc, vc = codes.clone(), codes.clone()
        ks, vs = (torch.full((1, 1, 1), 7.0, device="cuda") for _ in range(2))
        fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, ref.ints([3]), freq, block=16)
        return vc[0, 0, :3].double(), float(vs)

    y, s = one(v)
    assert s == 2.0 ** -100 and bool((y == 0).all())
    v[0, 0, 0, 0], v[0, 0, 1, 1], v[0, 0, 2, 2], v[0, 0, 0, 3] = math.inf, -math.inf, math.nan, 3.0
    y, s = one(v)
    assert s == r8.least_scale(3.0) and y[0, 3] * s == 3.0
    assert bool(torch.isnan(torch.stack([y[0, 0], y[1, 1], y[2, 2]])).all()) and int(torch.isnan(y).sum()) == 3


def test_own_positions_factor_and_in_place_q():
    g = ref.gen(1005)
    pos = torch.randint(-5000, 1 << 20, (2, 9), generator=g, device="cuda", dtype=torch.int32)
    run(g, 2, 4, 2, 9, 50, 128, 128, 64, False, "bhnd", [30, 50], factor=-1.25, positions=pos)
    run(g, 2, 4, 2, 9, 50, 128, 128, 64, True, "bhnd", [30, 50], positions=pos[0])
    q, k, v = (ref.draw(g, 2, h, 9, 64) for h in (4, 2, 2))
    freq, _ = fa_rope_frequencies(64)
    kc, ks = r8.cache(g, 2, 2, 50, 64, 64)
    vc, vs = r8.cache(g, 2, 2, 50, 64, 64)
    want = fa_rope(q, None, freq, pos)[0]
    got = fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, ref.ints([9, 50]), freq, pos, q_out=q)
    assert got is q and torch.equal(q, want)


def test_twice_the_same_and_in_two_parts():
    """The same rows again change nothing; a run in two calls may only differ by the rounding of the first part."""
    g = ref.gen(1006)
    q, k, v = (ref.draw(g, 1, 2, 50, 64) for _ in range(3))
    freq, _ = fa_rope_frequencies(64)
    kc, ks = r8.cache(g, 1, 2, 128, 64, 32)
    vc, vs = r8.cache(g, 1, 2, 128, 64, 32)
    fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, ref.ints([70]), freq, block=32)
    a = [t.clone() for t in (kc, ks, vc, vs)]
    fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, ref.ints([70]), freq, block=32)
    for x, y in zip(a, (kc, ks, vc, vs)):
        assert torch.equal(x.view(torch.uint8) if x.dtype == r8.E4M3 else x, y.view(torch.uint8) if y.dtype == r8.E4M3 else y)
    fa_rope_append_fp8(q[:, :, :31], k[:, :, :31], v[:, :, :31], kc, vc, ks, vs, ref.ints([51]), freq, block=32)
    fa_rope_append_fp8(q[:, :, 31:], k[:, :, 31:], v[:, :, 31:], kc, vc, ks, vs, ref.ints([70]), freq, block=32)
    assert torch.equal(ks, a[1]) and torch.equal(vs, a[3])
    off = (r8.values(vc, vs, 32) - r8.values(a[2], a[3], 32)).abs()
    s = vs.double().repeat_interleave(32, -1)[..., None]
    assert bool((off <= 2.0 ** -9 * s)[:, :, 20:70].all())  # a shift of exponents: one of e4m3's least steps at most


def test_graph_and_other_stream():
    g = ref.gen(1007)
    q, k, v = (ref.draw(g, 2, h, 1, 128) for h in (8, 2, 2))
    freq, _ = fa_rope_frequencies(128)
    kc, ks = r8.cache(g, 2, 2, 300, 128, 64)
    vc, vs = r8.cache(g, 2, 2, 300, 128, 64)
    lens = ref.ints([200, 300])
    state = [t.clone() for t in (kc, ks, vc, vs)]
    want = fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, lens, freq)
    after = [t.clone() for t in (kc, ks, vc, vs)]
    back = lambda: [t.copy_(x) for t, x in zip((kc, ks, vc, vs), state)]  # noqa: E731

    def same(out):
        assert torch.equal(out, want)
        for t, x in zip((kc, ks, vc, vs), after):
            assert torch.equal(t.view(torch.uint8) if t.dtype == r8.E4M3 else t, x.view(torch.uint8) if x.dtype == r8.E4M3 else x)

    back()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, lens, freq, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same(out)
    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, lens, freq)
    back()
    graph.replay()
    same(out)
