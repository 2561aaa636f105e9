"""C-ABI boundary of the operators on a cache held in 8 bits and of the
verification, on the CPU: every refusal happens on the host before any CUDA
call, so fake device addresses do.  And the plain forms that the GPU tests
compare with, against a library routine and hand-worked cases."""
import ctypes
import math

import pytest
import torch

import fp8_cache_refs as r8
from exact_attention_48_gb300 import build as fa_build
from exact_attention_48_gb300.binding import library

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return library()


def at(n):
    """A fake, aligned device address; each n a gigabyte from the next."""
    return (1 << 40) + (n << 30)


def st(B, H, N, d):
    return s3(H * N * d, N * d, d)


def s3(*v):
    return (ctypes.c_int64 * 3)(*v)


def append(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), qo=at(3), kc=at(4), vc=at(5), ks=at(6), vs=at(7), lens=at(8), pos=at(9),
             pos_b=10, freq=at(10), B=2, H=4, Hkv=2, N=10, Nk=100, d=64, rot=64, inter=0, factor=1.0, block=64)
    a.update(kw)
    B, H, Hkv, N, Nk, d = (max(1, a[x]) for x in ("B", "H", "Hkv", "N", "Nk", "d"))
    sq, sk, sc = st(B, H, N, d), st(B, Hkv, N, d), st(B, Hkv, Nk, d)
    return lib.fa_rope_append_fp8(a["q"], sq, a["k"], sk, a["v"], sk, a["qo"], a.get("sqo", sq), a["kc"],
                                  a.get("skc", sc), a["vc"], a.get("svc", sc), a["ks"], a["vs"], a["lens"], a["pos"],
                                  a["pos_b"], a["freq"], a["B"], a["H"], a["Hkv"], a["N"], a["Nk"], a["d"], a["rot"],
                                  a["inter"], a["factor"], a["block"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(N=0), INVALID), (dict(Nk=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=0), INVALID), (dict(inter=2), INVALID),
    (dict(factor=math.inf), INVALID), (dict(block=0), INVALID), (dict(block=48), UNSUPPORTED),
    (dict(block=256), UNSUPPORTED), (dict(q=0), INVALID), (dict(v=0), INVALID), (dict(kc=0), INVALID),
    (dict(ks=0), INVALID), (dict(vs=0), INVALID), (dict(ks=at(6) + 2), INVALID), (dict(lens=0), INVALID),
    (dict(lens=at(8) + 2), INVALID), (dict(freq=0), INVALID), (dict(pos=at(9) + 1), INVALID), (dict(pos_b=-1), INVALID),
    (dict(kc=at(4) + 8), INVALID), (dict(skc=s3(12800, 6400, 72)), INVALID), (dict(skc=s3(12800, 6400, 65)), INVALID),
    (dict(skc=s3(12800, 6400, 32)), INVALID), (dict(vc=at(4)), INVALID), (dict(vc=at(4) + 64), INVALID),
    (dict(vs=at(6)), INVALID), (dict(ks=at(4) + 64), INVALID), (dict(ks=at(1)), INVALID), (dict(qo=at(0) + 128), INVALID),
    (dict(qo=at(1)), INVALID), (dict(kc=at(2)), INVALID), (dict(lens=at(7)), INVALID), (dict(freq=at(5)), INVALID),
    (dict(pos=at(6)), INVALID), (dict(B=1 << 16, N=1 << 15), INVALID),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code


def tree(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), ks=at(3), vs=at(4), o=at(5), lse=at(6), par=at(7), par_b=5, lens=at(8), B=2, H=4,
             Hkv=2, Nt=5, Nk=3000, d=64, block=32, scale=0.125, ws=at(9), ws_bytes=1 << 29)
    a.update(kw)
    B, H, Hkv, Nt, Nk, d = (max(1, a[x]) for x in ("B", "H", "Hkv", "Nt", "Nk", "d"))
    sq, sk = st(B, H, Nt, d), st(B, Hkv, Nk, d)
    return lib.fa_fwd_tree_fp8(a["q"], sq, a["k"], a.get("sk", sk), a["v"], sk, a["ks"], a["vs"], a["o"],
                               a.get("so", sq), a["lse"], a["par"], a["par_b"], a["lens"], a["B"], a["H"], a["Hkv"],
                               a["Nt"], a["Nk"], a["d"], a["block"], a["scale"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(H=5), INVALID), (dict(Nt=0), INVALID), (dict(Nt=129), INVALID),
    (dict(Nk=0), INVALID), (dict(d=32), UNSUPPORTED), (dict(block=1), UNSUPPORTED), (dict(block=-16), INVALID),
    (dict(scale=math.nan), INVALID), (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(ks=0), INVALID),
    (dict(vs=at(4) + 1), INVALID), (dict(o=0), INVALID), (dict(lse=0), INVALID), (dict(par=at(7) + 2), INVALID),
    (dict(par_b=-5), INVALID), (dict(lens=at(8) + 2), INVALID), (dict(k=at(1) + 8), INVALID),
    (dict(sk=s3(384000, 192000, 24)), INVALID), (dict(so=s3(1280, 320, 32)), INVALID), (dict(o=at(0)), INVALID),
    (dict(o=at(1)), INVALID), (dict(o=at(3)), INVALID), (dict(lse=at(5) + 64), INVALID), (dict(lse=at(4)), INVALID),
    (dict(lse=at(7)), INVALID), (dict(lens=at(6)), INVALID), (dict(ws_bytes=1000), WORKSPACE),
    (dict(ws=at(9) + 64), INVALID), (dict(ws=at(4)), INVALID), (dict(ws=at(5)), INVALID),
])
def test_tree_refuses(lib, kw, code):
    assert tree(lib, **kw) == code


def test_tree_workspace(lib):
    assert lib.fa_tree_fp8_workspace_bytes(2, 4, 2, 5, 3000, 64) > 0
    assert lib.fa_tree_fp8_workspace_bytes(2, 4, 2, 5, 1000, 64) == 0      # short caches are not cut
    for bad in ((0, 4, 2, 5, 3000, 64), (2, 5, 2, 5, 3000, 64), (2, 4, 2, 129, 3000, 64), (2, 4, 2, 5, 3000, 80)):
        assert lib.fa_tree_fp8_workspace_bytes(*bad) == 0


def compact(lib, **kw):
    a = dict(k=at(0), v=at(1), ks=at(2), vs=at(3), ko=at(4), vo=at(5), kso=at(6), vso=at(7), kept=at(8), kb=40, kh=20,
             base=at(9), B=2, Hkv=2, Nk=100, Nout=50, M=20, d=64, block=16)
    a.update(kw)
    B, Hkv, Nk, Nout, d = (max(1, a[x]) for x in ("B", "Hkv", "Nk", "Nout", "d"))
    sk, so = st(B, Hkv, Nk, d), st(B, Hkv, Nout, d)
    return lib.fa_cache_compact_fp8(a["k"], a.get("sk", sk), a["v"], sk, a["ks"], a["vs"], a["ko"], a.get("sko", so),
                                    a["vo"], so, a["kso"], a["vso"], a["kept"], a["kb"], a["kh"], a["base"], a["B"],
                                    a["Hkv"], a["Nk"], a["Nout"], a["M"], a["d"], a["block"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(Nk=0), INVALID), (dict(Nout=0), INVALID), (dict(M=0), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(block=8), UNSUPPORTED), (dict(k=0), INVALID), (dict(vo=0), INVALID),
    (dict(ks=0), INVALID), (dict(vso=0), INVALID), (dict(kept=0), INVALID), (dict(kept=at(8) + 2), INVALID),
    (dict(kb=-1), INVALID), (dict(kh=-1), INVALID), (dict(base=at(9) + 2), INVALID), (dict(ko=at(4) + 4), INVALID),
    (dict(sko=s3(6400, 3200, 33)), INVALID), (dict(sko=s3(6400, 3200, 32)), INVALID), (dict(ko=at(0)), INVALID),
    (dict(vo=at(0)), INVALID), (dict(ko=at(5)), INVALID), (dict(kso=at(2)), INVALID), (dict(kso=at(7)), INVALID),
    (dict(kso=at(8)), INVALID), (dict(kso=at(4)), INVALID), (dict(vso=at(1)), INVALID), (dict(kept=at(4)), INVALID),
    (dict(base=at(6)), INVALID), (dict(ks=at(5)), INVALID),
    # in place but for one output
    (dict(ko=at(0), vo=at(1), kso=at(2), vso=at(3)), INVALID),
    (dict(ko=at(0), vo=at(1), kso=at(2), Nout=100), INVALID),
    (dict(B=1 << 11, Hkv=1 << 11, M=1 << 15), INVALID),
])
def test_compact_refuses(lib, kw, code):
    assert compact(lib, **kw) == code


def verify(lib, **kw):
    a = dict(par=at(0), par_b=8, tok=at(1), tok_b=8, t=at(2), tb=8000, tn=1000, q=at(3), qb=8000, qn=1000, u=at(4), ub=8,
             acc=at(5), cnt=at(6), nxt=at(7), B=2, Nt=8, V=1000)
    a.update(kw)
    return lib.fa_tree_verify(a["par"], a["par_b"], a["tok"], a["tok_b"], a["t"], a["tb"], a["tn"], a["q"], a["qb"],
                              a["qn"], a["u"], a["ub"], a["acc"], a["cnt"], a["nxt"], a["B"], a["Nt"], a["V"], None)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=1 << 24), dict(Nt=0), dict(Nt=129), dict(V=0), dict(V=(1 << 30) + 1), dict(par=0), dict(tok=0),
    dict(t=0), dict(u=0), dict(acc=0), dict(cnt=0), dict(nxt=0), dict(par=at(0) + 1), dict(t=at(2) + 2),
    dict(q=at(3) + 2), dict(u=at(4) + 3), dict(acc=at(5) + 2), dict(par_b=-1), dict(tok_b=-1), dict(tb=-1), dict(tn=-1),
    dict(qb=-1), dict(qn=-1), dict(ub=-1), dict(tb=1 << 39), dict(acc=at(0)), dict(cnt=at(5)), dict(nxt=at(6)),
    dict(nxt=at(2) + 4000), dict(cnt=at(3)), dict(acc=at(4)), dict(nxt=at(1)),
])
def test_verify_refuses(lib, kw):
    assert verify(lib, **kw) == INVALID


# ---------------------------------------------------------------- the plain forms


def test_plain_rounding_is_the_library_routine():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40000, generator=g) * torch.exp2(torch.randint(-14, 8, (40000,), generator=g).float())
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    near = codes[torch.isfinite(codes)].sort().values
    x = torch.cat([x.clamp(-448, 448), near, (near[1:] + near[:-1]) / 2])
    assert torch.equal(r8.round_e4m3(x.double()), x.to(torch.float8_e4m3fn).double())
    assert bool(torch.isnan(r8.round_e4m3(torch.tensor([math.inf, -math.inf, math.nan]).double())).all())


@pytest.mark.parametrize("a,s", [(0.0, 2.0 ** -100), (448.0, 1.0), (448.1, 2.0), (447.9, 1.0), (224.0, 0.5),
                                 (1.0, 2.0 ** -8), (2.0 ** -120, 2.0 ** -100), (3.3e38, 2.0 ** 120), (1.75, 2.0 ** -8),
                                 (1.76, 2.0 ** -7)])
def test_plain_scale(a, s):
    assert r8.least_scale(a) == s


def test_plain_verify_by_hand():
    # two children of the root: p = (.2, .5, .3), q = (.6, .2, .2); token 0 is rejected at u = .4 (.4 * .6 >= .2),
    # R = (0, .3, .1), S = .4; token 1: .9 * .2 * .4 < .3
    p, q = [[0.2, 0.5, 0.3]] * 3, [[0.6, 0.2, 0.2]] * 3
    assert r8.verify([-1, 0, 0], [0, 0, 1], p, q, [0.1, 0.4, 0.9]) == ([0, 2], 0)
    assert r8.verify([-1, 0, 0], [0, 0, 1], p, q, [0.2, 0.4, 0.9]) == ([0, 2], 1)
    assert r8.verify([-1, 0, 0], [0, 0, 1], p, q, [0.1, 0.3, 0.9]) == ([0, 1], 0)
    # both rejected: R = (0, .3, .1), then max(R - .4 q, 0) = (0, .22, .02)
    assert r8.verify([-1, 0, 0], [0, 0, 0], p, q, [0.91, 0.4, 0.0]) == ([0], 1)
    assert r8.verify([-1, 0, 0], [0, 0, 0], p, q, [0.92, 0.4, 0.0]) == ([0], 2)
    # chosen for certain: token 1 is rejected at u >= .5, its mass gone
    assert r8.verify([-1, 0], [0, 1], p, None, [0.39, 0.5]) == ([0], 0)
    assert r8.verify([-1, 0], [0, 1], p, None, [0.41, 0.5]) == ([0], 2)
    assert r8.verify([-2, 0], [0, 1], p, None, [0.41, 0.1]) == ([], -1)
