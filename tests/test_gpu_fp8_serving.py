"""The operators on a cache held in 8 bits together, as a server calls them: the
step of the project's front page run as it stands there, each call beside its
64-bit definition on the same codes (the bounds are those of the single calls);
the same in a graph; caches whose offsets pass 32 bits; two caches on two streams;
bounded waits."""
import ctypes
import glob
import math
import os
import re

import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
import exact_attention_48_gb300 as fa
from exact_attention_48_gb300 import build as fa_build
from test_gpu_fp8_append import check_k, check_v
from test_gpu_fp8_compact import check as check_compact
from test_gpu_fp8_tree import check as check_tree
from test_gpu_verify import check as check_verify

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
V = 500


def example():
    with open(glob.glob(os.path.join(ROOT, "README*"))[0], encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "fa_fwd_tree_fp8" in b)


class Held:
    """The package, each call of the step held against its definition."""

    def __init__(self):
        self.seen = []

    def fa_rope_append_fp8(self, q, k, v, kc, vc, ks, vs, lens, freq, positions):
        before = [t.clone() for t in (kc, ks, vc, vs)]
        out = fa.fa_rope_append_fp8(q, k, v, kc, vc, ks, vs, lens, freq, positions)
        rot = 2 * freq.numel()
        y, mag = ref.rope(q, positions, freq, rot, False, 1.0)
        fine = torch.isfinite(y)
        err = (out.double() - y).abs()[fine]
        assert bool((err <= (2.0 ** -8 * y.abs() + 2.0 ** -20 * mag + 1e-30)[fine]).all())
        x, mag = ref.rope(k, positions, freq, rot, False, 1.0)
        for b, n in enumerate(lens.tolist()):
            for h in range(kc.shape[1]):
                if bool(torch.isfinite(x[b, h]).all()):
                    check_k(kc[b, h], ks[b, h], x[b, h], mag[b, h], n, before[0][b, h], before[1][b, h], 64, 1.0, f"b{b} h{h}")
                check_v(vc[b, h], vs[b, h], v[b, h], n, before[2][b, h], before[3][b, h], 64, f"b{b} h{h}")
        self.seen.append("append")
        return out

    def fa_fwd_tree_fp8(self, q, kc, vc, ks, vs, parents, lens):
        o, lse = fa.fa_fwd_tree_fp8(q, kc, vc, ks, vs, parents, lens)
        B, H, Nt, d = q.shape
        G = H // kc.shape[1]
        kv, vv = r8.values(kc, ks, 64), r8.values(vc, vs, 64)
        for b, n in enumerate(lens.tolist()):
            for h in range(kc.shape[1]):
                heads = slice(h * G, h * G + G)
                check_tree(o[b, heads], lse[b, heads], q[b, heads].nan_to_num(0.0), kv[b, h], vv[b, h], parents[b].tolist(),
                           n, Nt, 1 / math.sqrt(d), f"b{b} h{h}", (vc[b, h], vs[b, h], 64))
        self.seen.append("attend")
        return o, lse

    def fa_tree_verify(self, parents, tokens, target, draft, u):
        got = fa.fa_tree_verify(parents, tokens, target, draft, u)
        check_verify(parents, tokens, target, draft, u, got)
        self.seen.append("verify")
        return got

    def fa_cache_compact_fp8(self, kc, vc, ks, vs, accepted, base):
        before = [t.clone() for t in (kc, vc, ks, vs)]
        out = fa.fa_cache_compact_fp8(kc, vc, ks, vs, accepted, base)
        check_compact(before[0], before[2], kc, ks, before[0], before[2], accepted, base.tolist(), 64, "k")
        check_compact(before[1], before[3], vc, vs, before[1], before[3], accepted, base.tolist(), 64, "v")
        self.seen.append("compact")
        return out


def setting(seed, B, H, Hkv, Nk, Nt, d, used):
    """Names that the step needs: a cache of `used` rows a sequence, stored by the library itself."""
    g = ref.gen(seed)
    names = {"torch": torch, "fa": fa, "d": d, "freq": fa.fa_rope_frequencies(d)[0]}
    for kind in ("k", "v"):
        names[kind + "c"] = torch.full((B, Nk, Hkv, d), 0x7F, device="cuda", dtype=torch.uint8).view(r8.E4M3).transpose(1, 2)
        names[kind + "s"] = torch.full((B, Hkv, -(-Nk // 64)), math.nan, device="cuda")
    N = max(used)
    pos = ref.ints([[i - (N - n) for i in range(N)] for n in used])
    q, k, v = (ref.draw(g, B, h, N, d) for h in (H, Hkv, Hkv))
    fa.fa_rope_append_fp8(q, k, v, names["kc"], names["vc"], names["ks"], names["vs"], ref.ints(used), names["freq"], pos)
    table = torch.randn(H * d, V, generator=g, device="cuda") * 0.5
    names["probs"] = lambda o: torch.softmax(o.transpose(1, 2).flatten(2).float() @ table, -1)
    return g, names


def draws(g, B, H, Hkv, Nt, d, lens, parents, depth):
    """One step's inputs: drafted tokens likely under the draft, lens with the new rows counted."""
    draft = torch.softmax(torch.randn(B, Nt, V, generator=g, device="cuda") * 0.5, -1)
    tokens = torch.randint(0, V, (B, Nt), generator=g, device="cuda", dtype=torch.int32)
    q, k, v = (ref.draw(g, B, h, Nt, d) for h in (H, Hkv, Hkv))
    return {"q": q, "k": k, "v": v, "lens": lens + Nt, "positions": ref.ints(depth) + lens[:, None],
            "parents": ref.ints(parents), "tokens": tokens, "draft": draft, "u": torch.rand(B, Nt, generator=g, device="cuda")}


def depths(parents):
    out = []
    for row in parents:
        dep = [0] * len(row)
        for i, p in enumerate(row):
            dep[i] = dep[p] + 1 if 0 <= p < i else 0
        out.append(dep)
    return out


PARENTS = [[-1, 0, 0, 1, 1, 2, 3, 5], [-1, 0, 0, 0, 0, 4, -2, -2], [-2, -1, 0, 1, 2, 3, 3, 6]]


@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 4, 2), (128, 8, 1), (64, 6, 3)])
def test_the_step(d, H, Hkv):
    B, Nk, Nt = 3, 400, 8
    g, names = setting(700 + d + H, B, H, Hkv, Nk, Nt, d, [130, 63, 200])
    names["fa"], lens = Held(), ref.ints([130, 63, 200])
    code, accepted = compile(example(), "example", "exec"), 0
    for step in range(6):
        names.update(draws(g, B, H, Hkv, Nt, d, lens, PARENTS, depths(PARENTS)))
        exec(code, names)
        assert fa.fa_device_status() == 0
        counts = names["counts"].tolist()
        assert counts[2] == 0 and counts[0] >= 1 and names["lens"].tolist() == [n + c for n, c in zip(lens.tolist(), counts)]
        assert int(names["token"][2]) == -1
        accepted += sum(counts)
        lens = names["lens"]
    assert names["fa"].seen == ["append", "attend", "verify", "compact"] * 6


def test_the_step_in_a_graph():
    """Captured once and replayed on new inputs: the same bits as the calls made one by one."""
    B, H, Hkv, Nk, Nt, d = 3, 16, 2, 2000, 8, 128
    used = [1500, 63, 200]
    g, names = setting(710, B, H, Hkv, Nk, Nt, d, used)
    code = compile(example(), "example", "exec")
    twin = dict(names)
    for n in ("kc", "vc", "ks", "vs"):
        twin[n] = names[n].clone(memory_format=torch.preserve_format)
    static = draws(ref.gen(711), B, H, Hkv, Nt, d, ref.ints(used), PARENTS, depths(PARENTS))
    save = {n: names[n].clone(memory_format=torch.preserve_format) for n in ("kc", "vc", "ks", "vs")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        names.update(static)
        exec(code, names)                       # (warm-up)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    names.update(static)
    with torch.cuda.graph(graph):
        exec(code, names)
    out = {n: names[n] for n in ("o", "lse", "accepted", "counts", "token", "lens")}
    for n, t in save.items():
        names[n].copy_(t)
    lens = ref.ints(used)
    for step in range(4):
        new = draws(g, B, H, Hkv, Nt, d, lens, PARENTS, depths(PARENTS))
        for n, t in new.items():
            static[n].copy_(t)
        graph.replay()
        twin.update(new)
        exec(code, twin)
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], twin[n]), (step, n)
        for n in ("kc", "vc"):
            assert torch.equal(names[n].view(torch.uint8), twin[n].view(torch.uint8)), (step, n)
        for n in ("ks", "vs"):
            assert torch.equal(names[n].nan_to_num(), twin[n].nan_to_num()), (step, n)
        lens = out["lens"].clone()
    assert fa.fa_device_status() == 0


def test_two_caches_on_two_streams():
    B, H, Hkv, Nk, Nt, d = 2, 8, 2, 3000, 8, 128
    code, parents = compile(example(), "example", "exec"), PARENTS[:2]
    runs = []
    for seed in (720, 721):
        g, names = setting(seed, B, H, Hkv, Nk, Nt, d, [2500, 700])
        steps, lens = [], ref.ints([2500, 700])
        for _ in range(3):
            steps.append(draws(g, B, H, Hkv, Nt, d, lens, parents, depths(parents)))
        runs.append((names, steps))

    def go(names, steps):
        names, lens = dict(names), None
        for n in ("kc", "vc", "ks", "vs"):
            names[n] = names[n].clone(memory_format=torch.preserve_format)
        outs = []
        for s in steps:
            names.update(s)
            if lens is not None:
                names["lens"] = lens + Nt
            exec(code, names)
            lens = names["lens"]
            outs += [names[n] for n in ("o", "lse", "accepted", "token")]
        return outs + [names[n].view(torch.uint8) for n in ("kc", "vc")]

    alone = [go(*r) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        both = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                both.append(go(*r))
        torch.cuda.synchronize()
        for a, z in zip(alone, both):
            assert all(torch.equal(x, y) for x, y in zip(a, z))
    assert fa.fa_device_status() == 0


@pytest.mark.parametrize("far", ["heads", "rows", "sequences"])
def test_offsets_past_32_bits(far):
    """Caches spread over more than 2^32 elements: the same bits as packed ones."""
    B, H, Hkv, Nk, Nt, d = 2, 6, 3, 4500, 8, 64
    Bs, Hs, Ns = {"heads": (64 * Nk, (1 << 31) + 4096, 64), "rows": (64 * Hkv, 64, 1 << 20),
                  "sequences": (1 << 33, 64 * Nk, 64)}[far]
    size = (B - 1) * Bs + (Hkv - 1) * Hs + (Nk - 1) * Ns + d
    assert size > 1 << 32
    g, names = setting(730, B, H, Hkv, Nk, Nt, d, [4400, 2100])
    wide = dict(names)
    for n in ("kc", "vc"):
        t = torch.empty(size, dtype=torch.uint8, device="cuda").as_strided((B, Hkv, Nk, d), (Bs, Hs, Ns, 1)).view(r8.E4M3)
        t.copy_(names[n])
        wide[n] = t
    for n in ("ks", "vs"):
        wide[n] = names[n].clone()
    parents = PARENTS[:2]
    inputs = draws(g, B, H, Hkv, Nt, d, ref.ints([4400, 2100]), parents, depths(parents))
    code = compile(example(), "example", "exec")
    for x in (names, wide):
        x.update(inputs)
        exec(code, x)
    assert fa.fa_device_status() == 0
    for n in ("o", "lse", "accepted", "token"):
        assert torch.equal(names[n], wide[n]), n
    for n in ("kc", "vc"):
        assert torch.equal(names[n].contiguous().view(torch.uint8), wide[n].contiguous().view(torch.uint8)), n
    for n in ("ks", "vs"):
        assert torch.equal(names[n].nan_to_num(), wide[n].nan_to_num()), n
    kept = torch.arange(0, 4500, 2, device="cuda", dtype=torch.int32).expand(B, -1).contiguous()
    for x in (names, wide):
        fa.fa_cache_compact_fp8(x["kc"], x["vc"], x["ks"], x["vs"], kept)
    assert torch.equal(names["kc"][:, :, :2000].contiguous().view(torch.uint8), wide["kc"][:, :, :2000].contiguous().view(torch.uint8))


# ---------------------------------------------------------------- bounded waits, see test_gpu_cache_timeout.py
FA_OK, FA_ERR_DEVICE_TIMEOUT = 0, 5


@pytest.fixture(scope="module")
def stall():
    lib = ctypes.CDLL(fa_build.build_variant("stalltest"))
    vp, i, f, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64, ctypes.c_size_t
    lib.fa_fwd_tree_fp8.argtypes = [vp] * 12 + [i64, vp] + [i] * 7 + [f, vp, sz, vp]
    lib.fa_device_status.argtypes = [vp]
    lib.fa_debug_last_wait_site.argtypes = []
    return lib


# 16 and 32 columns and 128 lanes: one unit, a cut unit, many units a run, a tree's table in the first tile
@pytest.mark.parametrize("B,H,Hkv,Nt,Nk,d", [
    (1, 2, 2, 5, 300, 128), (1, 8, 1, 1, 20000, 64), (70, 4, 4, 3, 500, 64), (1, 4, 1, 7, 20000, 128), (70, 8, 2, 8, 500, 64),
    (2, 8, 2, 64, 3000, 128), (1, 4, 1, 33, 20000, 64), (70, 8, 2, 10, 500, 128), (1, 1, 1, 40, 100, 64)])
def test_bounded_waits(stall, B, H, Hkv, Nt, Nk, d):
    g = ref.gen(740)
    q = ref.draw(g, B, H, Nt, d)
    k, ks = r8.cache(g, B, Hkv, Nk, d, 64)
    v, vs = r8.cache(g, B, Hkv, Nk, d, 64)
    par = ref.ints(list(range(-1, Nt - 1)))
    st = [(ctypes.c_int64 * 3)(*t.stride()[:3]) for t in (q, k, v)]
    a = [ctypes.addressof(x) for x in st]
    s = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        o, lse = torch.zeros_like(q), torch.zeros(B, H, Nt, device="cuda")
        rc = stall.fa_fwd_tree_fp8(q.data_ptr(), a[0], k.data_ptr(), a[1], v.data_ptr(), a[2], ks.data_ptr(), vs.data_ptr(),
                                   o.data_ptr(), a[0], lse.data_ptr(), par.data_ptr(), 0, None, B, H, Hkv, Nt, Nk, d, 64,
                                   0.01, None, 0, s)
        assert rc == FA_OK
        torch.cuda.synchronize()                                     # every kernel has returned
        site = stall.fa_debug_last_wait_site()
        assert stall.fa_device_status(s) == FA_ERR_DEVICE_TIMEOUT and site > 0
        assert stall.fa_device_status(s) == FA_OK                    # reported once
    o, lse = fa.fa_fwd_tree_fp8(q, k, v, ks, vs, par)
    assert fa.fa_device_status() == FA_OK and bool(torch.isfinite(lse).all())
