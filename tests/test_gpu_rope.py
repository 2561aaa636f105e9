"""Rotary positions (fa_rope, fa_rope_bwd, fa_rope_append) against the 64-bit
rotation.

Bound per element: the result is rounded once to bf16 (at most 2^-8 of it);
cos and sin carry the fp32 rounding of the reduced angle (2^-25 half turns,
about 1e-7) and of sincospi and the products (a few 2^-24), together below
2^-20 of |x1| + |x2| and the factor.  Past rot the columns are copies.
"""
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import FaError, fa_rope, fa_rope_append, fa_rope_bwd, fa_rope_frequencies

pytestmark = pytest.mark.gpu


def _bound(y, mag, factor):
    return 2.0 ** -8 * y.abs() + 2.0 ** -20 * abs(factor) * mag + 1e-30


def _check(got, x, pos, freq, interleaved, factor, sign, what):
    rot = 2 * freq.numel()
    y, mag = ref.rope(x, pos, freq, rot, interleaved, factor, sign)
    err = (got.double() - y).abs()
    assert bool((err <= _bound(y, mag, factor)).all()), f"{what}: max err {float(err.max()):.3e}"
    assert torch.equal(got[..., rot:], x[..., rot:]), f"{what}: columns past rot"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hkv,N,d,rot,layout", [
    (1, 1, 1, 1, 64, 64, "bhnd"),
    (2, 4, 2, 33, 128, 128, "bhnd"),
    (3, 5, 1, 257, 64, 16, "bnhd"),
    (1, 3, 3, 1001, 128, 48, "pitch"),
    (2, 7, 0, 65, 128, 112, "bnhd"),
    (17, 2, 2, 2, 64, 32, "bhnd"),
])
def test_rope_and_gradient(B, H, Hkv, N, d, rot, layout, interleaved):
    g = ref.gen(B + 10 * H + N)
    q = ref.draw(g, B, H, N, d, layout)
    k = ref.draw(g, B, Hkv, N, d, layout) if Hkv else None
    freq, factor = fa_rope_frequencies(rot, 10000.0, "by_parts", 8.0)
    pos = torch.randint(-5000, 1 << 20, (B, N), generator=g, device="cuda", dtype=torch.int32)
    for call, sign in ((fa_rope, 1.0), (fa_rope_bwd, -1.0)):
        a, b = call(q, k, freq, pos, interleaved, factor)
        _check(a, q, pos, freq, interleaved, factor, sign, "q")
        if Hkv:
            _check(b, k, pos, freq, interleaved, factor, sign, "k")
        else:
            assert b is None


def test_default_and_shared_positions():
    g = ref.gen(5)
    q, k = ref.draw(g, 3, 4, 130, 64), ref.draw(g, 3, 2, 130, 64)
    freq, _ = fa_rope_frequencies(64)
    n = torch.arange(130, dtype=torch.int32, device="cuda")
    a = fa_rope(q, k, freq)
    for pos in (n, n.expand(3, 130).contiguous(), n.expand(3, 130)):
        for x, y in zip(a, fa_rope(q, k, freq, pos)):
            assert torch.equal(x, y)
    _check(a[0], q, n.expand(3, 130), freq, False, 1.0, 1.0, "q")


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_packed_projection(interleaved):
    """q and k slices of one packed projection, rotated where they are; v untouched."""
    g = ref.gen(6)
    B, N, H, Hkv, d = 2, 77, 6, 2, 128
    packed = torch.randn(B, N, H + 2 * Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    before = packed.clone()
    view = packed.transpose(1, 2)
    q, k = view[:, :H], view[:, H:H + Hkv]
    freq, _ = fa_rope_frequencies(64)
    want = fa_rope(q, k, freq, None, interleaved)
    got = fa_rope(q, k, freq, None, interleaved, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(packed[:, :, H + Hkv:], before[:, :, H + Hkv:])
    # one q head, one k head beside it
    fa_rope(view[:, :1], view[:, 1:2], freq, q_out=view[:, :1], k_out=view[:, 1:2])


def test_far_positions_and_fast_frequencies():
    """Angles modulo a turn hold for every 32-bit position, also for frequencies above a radian per position and
    far below 2^-24 turns."""
    g = ref.gen(7)
    freq = torch.tensor([1.0, 3.0, 6.2831855, 100.5, 0.5, 1e-3, 1e-7, 1e-12], device="cuda")
    pos = ref.ints([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24, 123456789, 7]])
    q = ref.draw(g, 1, 2, 8, 64)
    out, _ = fa_rope(q, None, freq, pos)
    # 2^31 * f * 2^-64 per unit of the fixed-point step and f's 53-bit reference product: both far below 2^-20
    a = pos.double()[0, :, None] * freq.double()
    want, mag = ref.rope(q, pos, freq, 16, False, 1.0)
    # the fp64 reference's own angle error: 2^-53 |a| + the reduction's, on top of the bound
    slack = (2.0 ** -50 * a.abs().max()).item()
    err = (out.double() - want).abs()
    assert bool((err <= _bound(want, mag, 1.0) + slack * mag).all()), float(err.max())


def test_gradient_against_differences():
    """<dL/dy, (rope(x + h e) - rope(x - h e)) / 2h> equals dx_e: the map is linear, so with x = 0 and h = 1 the
    difference quotient is the rotated unit vector, exact but for its bf16 rounding (2^-8 per element)."""
    g = ref.gen(8)
    d, rot = 64, 32
    freq, factor = fa_rope_frequencies(rot, scaling="by_parts", factor=4.0)
    dy = ref.draw(g, 1, 1, d, d)
    pos = torch.full((1, d), 1234, dtype=torch.int32, device="cuda")
    eye = torch.eye(d, device="cuda", dtype=torch.bfloat16)[None, None]
    for inter in (False, True):
        rows, _ = fa_rope(eye, None, freq, pos, inter, factor)    # row e = rope(unit e)
        dx, _ = fa_rope_bwd(dy, None, freq, pos, inter, factor)
        num = dy[0, 0].double() @ rows[0, 0].double().T           # [token, e]
        tol = 2.0 ** -8 * (dy[0, 0].double().abs() @ rows[0, 0].double().abs().T) + 2.0 ** -8 * dx[0, 0].double().abs()
        assert bool(((dx[0, 0].double() - num).abs() <= tol + 1e-6).all())


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("B,H,Hkv,N,Nk,d,rot,interleaved", [
    (1, 2, 1, 1, 1, 64, 64, False), (4, 8, 2, 1, 200, 128, 128, False), (3, 4, 4, 37, 130, 128, 32, True),
    (2, 3, 1, 64, 64, 64, 48, False)])
def test_append(B, H, Hkv, N, Nk, d, rot, interleaved, layout):
    g = ref.gen(9 + N)
    q, k, v = ref.draw(g, B, H, N, d), ref.draw(g, B, Hkv, N, d, "bnhd"), ref.draw(g, B, Hkv, N, d, "pitch")
    kc, vc = ref.draw(g, B, Hkv, Nk, d, layout), ref.draw(g, B, Hkv, Nk, d, layout)
    k0, v0 = kc.clone(), vc.clone()
    # full, short (some rows before the cache), past the end, and far out on either side
    lens = ([Nk, N // 2, Nk + N // 2 + 1, -3] * B)[:B]
    freq, factor = fa_rope_frequencies(rot)
    qo = fa_rope_append(q, k, v, kc, vc, ref.ints(lens), freq, None, interleaved, factor)
    pos = torch.tensor([[n - N + i for i in range(N)] for n in lens], device="cuda")
    _check(qo, q, pos, freq, interleaved, factor, 1.0, "q")
    rot_k = fa_rope(k, None, freq, pos.to(torch.int32), interleaved, factor)[0]
    for b, n in enumerate(lens):
        for i in range(N):
            r = n - N + i
            if 0 <= r < Nk:
                k0[b, :, r], v0[b, :, r] = rot_k[b, :, i], v[b, :, i]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_append_own_positions_and_in_place():
    g = ref.gen(11)
    B, H, Hkv, N, Nk, d = 2, 4, 2, 5, 64, 128
    q, k, v = ref.draw(g, B, H, N, d), ref.draw(g, B, Hkv, N, d), ref.draw(g, B, Hkv, N, d)
    kc, vc = torch.zeros(B, Hkv, Nk, d, device="cuda", dtype=torch.bfloat16), torch.zeros(
        B, Hkv, Nk, d, device="cuda", dtype=torch.bfloat16)
    freq, _ = fa_rope_frequencies(d)
    pos = ref.ints([100, 101, 101, 102, 102])
    want, want_k = fa_rope(q, k, freq, pos)
    got = fa_rope_append(q, k, v, kc, vc, ref.ints([5, 64]), freq, pos, q_out=q)
    assert got is q and torch.equal(q, want)
    assert torch.equal(kc[0, :, :5], want_k[0]) and torch.equal(kc[1, :, 59:], want_k[1])
    assert torch.equal(vc[0, :, :5], v[0]) and not vc[0, :, 5:].any() and not kc[1, :, :59].any()


def test_offsets_past_2_31():
    """A cache whose element offsets pass 2^31: the last row of the last head."""
    B, Hkv, Nk, d = 1, 2, (1 << 23) + 64, 128
    kc = torch.zeros(B, Hkv, Nk, d, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    assert kc.numel() > 1 << 31
    g = ref.gen(12)
    q, k, v = (ref.draw(g, B, Hkv, 1, d) for _ in range(3))
    freq, _ = fa_rope_frequencies(d)
    fa_rope_append(q, k, v, kc, vc, ref.ints([Nk]), freq)
    want, _ = fa_rope(k, None, freq, ref.ints([Nk - 1]))
    assert torch.equal(kc[:, :, -1:], want) and torch.equal(vc[:, :, -1:], v)
    assert not kc[:, :, -2].any() and not vc[0, 0, :8].any()


def test_streams_and_capture():
    g = ref.gen(13)
    q, k = ref.draw(g, 2, 4, 300, 64), ref.draw(g, 2, 2, 300, 64)
    freq, _ = fa_rope_frequencies(64)
    want = fa_rope(q, k, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa_rope(q, k, freq, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa_rope(q, k, freq, q_out=a, k_out=b)
    q.copy_(ref.draw(g, 2, 4, 300, 64))
    graph.replay()
    torch.cuda.synchronize()
    want = fa_rope(q, k, freq)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_refusals():
    q = torch.zeros(1, 2, 8, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(1, 1, 8, 64, device="cuda", dtype=torch.bfloat16)
    freq, _ = fa_rope_frequencies(64)
    with pytest.raises(FaError):
        fa_rope(q, k, freq, q_out=torch.empty_like(k).expand(1, 2, 8, 64))   # heads share memory
    with pytest.raises(FaError):
        fa_rope(q, k, freq, k_out=q[:, :1])             # an output on an input
    with pytest.raises(FaError):
        fa_rope(q, k, freq, factor=math.inf)
    with pytest.raises(FaError):
        fa_rope(q, k, freq[:4])                          # rot = 8
    with pytest.raises(ValueError):
        fa_rope(q, k, freq, ref.ints([1, 2, 3]))
    with pytest.raises(ValueError):
        fa_rope(q, k, freq.double())
    with pytest.raises(ValueError):
        fa_rope(q, None, freq, k_out=k)
    with pytest.raises(TypeError):
        fa_rope(q.float(), k, freq)
    with pytest.raises(TypeError):
        fa_rope(q, k.cpu(), freq)
