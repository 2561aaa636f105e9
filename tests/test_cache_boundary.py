"""C-ABI boundary of the cache operators on the CPU: every refusal happens on
the host before any CUDA call, so fake device addresses do; and the host
function fa_rope_frequencies against its formulas."""
import ctypes
import math

import pytest
import torch

from exact_attention_48_gb300 import build as fa_build
from exact_attention_48_gb300 import fa_rope_frequencies
from exact_attention_48_gb300.binding import FaError, library

FA_OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return library()


def at(n):
    """A fake, aligned device address; each n a gigabyte from the next."""
    return (1 << 40) + (n << 30)


def st(B, H, N, d):
    return (ctypes.c_int64 * 3)(H * N * d, N * d, d)


def s3(*v):
    return (ctypes.c_int64 * 3)(*v)


def rope(lib, call="fa_rope", **kw):
    a = dict(q=at(0), k=at(1), qo=at(2), ko=at(3), pos=at(4), pos_b=10, freq=at(5), B=2, H=4, Hkv=2, N=10, d=64, rot=64,
             inter=0, factor=1.0)
    a.update(kw)
    sq, sk = st(a["B"], max(1, a["H"]), a["N"], a["d"]), st(a["B"], max(1, a["Hkv"]), a["N"], a["d"])
    return getattr(lib, call)(a["q"], a.get("sq", sq), a["k"], sk, a["qo"], a.get("sqo", sq), a["ko"],
                              a.get("sko", sk), a["pos"], a["pos_b"], a["freq"], a["B"], a["H"], a["Hkv"], a["N"],
                              a["d"], a["rot"], a["inter"], a["factor"], None)


@pytest.mark.parametrize("call", ["fa_rope", "fa_rope_bwd"])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=-1), INVALID), (dict(N=0), INVALID), (dict(d=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=80), INVALID), (dict(rot=24), UNSUPPORTED),
    (dict(inter=2), INVALID), (dict(factor=math.nan), INVALID), (dict(q=0), INVALID), (dict(freq=0), INVALID),
    (dict(k=0), INVALID), (dict(Hkv=0), INVALID), (dict(freq=at(5) + 2), INVALID), (dict(pos=at(4) + 1), INVALID),
    (dict(pos_b=-1), INVALID), (dict(q=at(0) + 8), INVALID), (dict(qo=at(0) + 128), INVALID), (dict(ko=at(0)), INVALID),
    (dict(ko=at(2)), INVALID), (dict(freq=at(2) + 64), INVALID), (dict(pos=at(3)), INVALID),
    (dict(sq=s3(2560, 640, 68)), INVALID), (dict(sqo=s3(2560, 640, 8)), INVALID), (dict(B=1 << 16, N=1 << 15), INVALID),
])
def test_rope_refuses(lib, call, kw, code):
    assert rope(lib, call, **kw) == code


def test_rope_append_refuses(lib):
    def call(**kw):
        a = dict(q=at(0), k=at(1), v=at(2), qo=at(3), kc=at(4), vc=at(5), lens=at(6), pos=None, freq=at(7), B=2, H=4,
                 Hkv=2, N=3, Nk=100, d=128, rot=128)
        a.update(kw)
        B, H, Hkv, N, Nk, d = (max(1, a[x]) for x in ("B", "H", "Hkv", "N", "Nk", "d"))
        sq, sk, sc = st(B, H, N, d), st(B, Hkv, N, d), st(B, Hkv, Nk, d)
        return lib.fa_rope_append(a["q"], sq, a["k"], sk, a["v"], sk, a["qo"], sq, a["kc"], a.get("skc", sc), a["vc"],
                                  sc, a["lens"], a["pos"], 0, a["freq"], a["B"], a["H"], a["Hkv"], a["N"], a["Nk"],
                                  a["d"], a["rot"], 0, 1.0, None)
    for kw in (dict(lens=None), dict(Hkv=0), dict(Nk=0), dict(kc=None), dict(vc=at(4) + 256), dict(kc=at(1)),
               dict(qo=at(2)), dict(lens=at(4) + 512), dict(lens=at(6) + 1), dict(skc=s3(25600, 12800, 64)),
               dict(freq=at(5))):
        assert call(**kw) == INVALID, kw
    assert call(rot=40) == UNSUPPORTED


def tree(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), o=at(3), lse=at(4), par=at(5), par_b=9, lens=at(6), B=2, H=4, Hkv=2, Nt=9,
             Nk=100, d=64, scale=0.1, ws=None, wsb=0)
    a.update(kw)
    B, H, Hkv, Nt, Nk, d = (max(1, a[x]) for x in ("B", "H", "Hkv", "Nt", "Nk", "d"))
    sq, sk = st(B, H, Nt, d), st(B, Hkv, Nk, d)
    return lib.fa_fwd_tree(a["q"], sq, a["k"], sk, a["v"], sk, a["o"], a.get("so", sq), a["lse"], a["par"], a["par_b"],
                           a["lens"], a["B"], a["H"], a["Hkv"], a["Nt"], a["Nk"], a["d"], a["scale"], a["ws"],
                           a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(Nt=0), INVALID), (dict(Nt=129), INVALID), (dict(H=5), INVALID), (dict(Hkv=0), INVALID), (dict(Nk=0), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(scale=math.inf), INVALID), (dict(par=None), INVALID), (dict(par=at(5) + 2), INVALID),
    (dict(par_b=-9), INVALID), (dict(lse=None), INVALID), (dict(lse=at(4) + 4), INVALID), (dict(o=at(0)), INVALID),
    (dict(o=at(2) + 1024), INVALID), (dict(lse=at(3)), INVALID), (dict(par=at(3)), INVALID), (dict(lens=at(4)), INVALID),
    (dict(lse=at(1)), INVALID), (dict(so=s3(2304, 576, 32)), INVALID), (dict(B=1 << 22, H=4), INVALID),
])
def test_tree_refuses(lib, kw, code):
    assert tree(lib, **kw) == code


def test_tree_workspace(lib):
    size = lib.fa_tree_workspace_bytes
    assert size(1, 8, 2, 7, 1 << 20, 128) % 256 == 0
    assert size(0, 8, 2, 7, 100, 128) == 0 and size(1, 8, 3, 7, 100, 128) == 0 and size(1, 8, 2, 129, 100, 128) == 0
    need = size(2, 4, 2, 9, 100000, 64)
    if need:
        assert tree(lib, Nk=100000, ws=at(8), wsb=need - 1) == WORKSPACE
        assert tree(lib, Nk=100000, ws=at(8) + 16, wsb=need) == INVALID
        assert tree(lib, Nk=100000, ws=at(3), wsb=need) == INVALID


def test_key_weights_refuses(lib):
    def call(**kw):
        a = dict(q=at(0), k=at(1), lse=at(2), wi=at(3), w=at(4), lens=at(5), B=2, H=4, Hkv=2, Nq=9, Nk=100, d=64,
                 causal=1, scale=0.1, ws=None, wsb=0)
        a.update(kw)
        B, H, Hkv, Nq, Nk, d = (max(1, a[x]) for x in ("B", "H", "Hkv", "Nq", "Nk", "d"))
        return lib.fa_key_weights(a["q"], st(B, H, Nq, d), a["k"], st(B, Hkv, Nk, d), a["lse"], a["wi"], a["w"],
                                  a["lens"], a["B"], a["H"], a["Hkv"], a["Nq"], a["Nk"], a["d"], a["causal"],
                                  a["scale"], a["ws"], a["wsb"], None)
    for kw in (dict(Nq=0), dict(Nk=0), dict(H=3), dict(causal=2), dict(scale=math.nan), dict(lse=None), dict(w=None),
               dict(w=at(0)), dict(w=at(1) + 1600), dict(w=at(2)), dict(w=at(5)), dict(w=at(3) + 16),
               dict(wi=at(3) + 4), dict(lens=at(5) + 3)):
        assert call(**kw) == INVALID, kw
    assert call(d=96) == UNSUPPORTED
    assert lib.fa_key_weights_workspace_bytes(2, 4, 2, 9, 100, 96) == 0
    need = lib.fa_key_weights_workspace_bytes(1, 4, 2, 4096, 500, 64)
    assert need % 256 == 0
    if need:
        sizes = dict(B=1, Nq=4096, Nk=500)
        assert call(ws=at(8), wsb=need - 1, **sizes) == WORKSPACE
        assert call(ws=at(8) + 16, wsb=need, **sizes) == INVALID
        assert call(ws=at(4), wsb=need, **sizes) == INVALID


def test_select_refuses(lib):
    def call(w=at(0), lens=at(1), kept=at(2), new=at(3), B=2, Hkv=2, Nk=100, keep=50, first=4, recent=8):
        return lib.fa_cache_select(w, lens, kept, new, B, Hkv, Nk, keep, first, recent, None)
    for kw in (dict(B=0), dict(Nk=0), dict(keep=0), dict(keep=101), dict(first=-1), dict(recent=-1),
               dict(first=45, recent=6), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), dict(w=None), dict(kept=None),
               dict(new=None), dict(new=at(1)), dict(kept=at(0) + 64), dict(new=at(2)), dict(w=at(0) + 4),
               dict(lens=at(1) + 2)):
        assert call(**kw) == INVALID, kw


def test_compact_refuses(lib):
    B, Hkv, Nk, M, d = 2, 2, 100, 10, 64
    s = st(B, Hkv, Nk, d)

    def call(k=at(0), v=at(1), w=at(2), ko=at(0), vo=at(1), wo=at(2), kept=at(3), kb=20, kh=10, base=None, nout=Nk, m=M,
             sk=s, d=d):
        return lib.fa_cache_compact(k, sk, v, s, w, ko, st(B, Hkv, nout, 64), vo, st(B, Hkv, nout, 64), wo, kept, kb,
                                    kh, base, B, Hkv, Nk, nout, m, d, None)
    for kw in (dict(k=None), dict(kept=None), dict(w=None), dict(wo=None), dict(m=0), dict(kb=-1), dict(kh=-1),
               dict(ko=at(5)), dict(vo=at(5)), dict(wo=at(5)), dict(ko=at(1), vo=at(0)),
               dict(ko=at(5), vo=at(5) + 128, wo=at(7)), dict(ko=at(5), vo=at(6), wo=at(2) + 16), dict(kept=at(0)),
               dict(base=at(1)), dict(base=at(3) + 1), dict(nout=50), dict(k=at(0) + 8), dict(nout=0)):
        assert call(**kw) == INVALID, kw
    assert call(d=32) == UNSUPPORTED


def test_rope_frequencies():
    rot = 64
    i = torch.arange(rot // 2, dtype=torch.float64)
    plain = 10000.0 ** (-2 * i / rot)

    def got(**kw):
        return fa_rope_frequencies(rot, device="cpu", **kw)

    def same(t, want):  # one rounding to fp32, and pow's own few 2^-53
        assert bool(((t.double() - want).abs() <= 2.0 ** -24 * want * 1.01).all())
    t, f = got()
    same(t, plain)
    assert f == 1.0
    t, f = got(scaling="linear", factor=4.0)
    same(t, plain / 4)
    t, f = got(scaling="base", factor=4.0)
    same(t, (10000.0 * 4.0 ** (rot / (rot - 2))) ** (-2 * i / rot))
    assert f == 1.0
    t, f = got(scaling="by_parts", factor=16.0, original_len=4096, fast_turns=32.0, slow_turns=1.0)
    turns = 4096 * plain / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    same(t, plain * keep + plain / 16 * (1 - keep))
    assert t[0] == 1.0 and abs(f - (1 + 0.1 * math.log(16.0))) <= 2.0 ** -23
    for kw in (dict(scaling="base", factor=0.5), dict(base=1.0), dict(base=math.inf),
               dict(scaling="by_parts", factor=2.0, original_len=0),
               dict(scaling="by_parts", factor=2.0, slow_turns=0.0),
               dict(scaling="by_parts", factor=2.0, fast_turns=1.0)):
        with pytest.raises(FaError):
            got(**kw)
    for rot_bad in (0, -2, 7):
        with pytest.raises(FaError):
            fa_rope_frequencies(rot_bad, device="cpu")
    with pytest.raises(FaError):
        fa_rope_frequencies(2, scaling="base", factor=2.0, device="cpu")
    with pytest.raises(ValueError):
        got(scaling="other")


def test_int_strides_past_64_bits_are_refused(lib):
    """Row strides whose products would not fit 64 bits."""
    for far in (1 << 39, 2 ** 62, 2 ** 63 - 1):
        assert rope(lib, pos_b=far) == INVALID and rope(lib, "fa_rope_bwd", pos_b=far) == INVALID
        assert tree(lib, par_b=far) == INVALID
        s = st(2, 2, 100, 64)
        for kb, kh in ((far, 10), (20, far)):
            assert lib.fa_cache_compact(at(0), s, at(1), s, None, at(4), s, at(5), s, None, at(3), kb, kh, None, 2, 2,
                                        100, 100, 10, 64, None) == INVALID
    s = st(1 << 10, 1 << 4, 100, 64)
    assert lib.fa_cache_compact(at(0), s, at(10), s, None, at(20), s, at(30), s, None, at(40), 0, 0, None, 1 << 10,
                                1 << 4, 100, 100, 1 << 30, 64, None) == INVALID
