"""The serving step of the project's front page, run as it stands there: a
drafted tree verified, its accepted branch kept, the keys weighed, the cache
cut back.  Two steps on one cache, beside a 64-bit program that takes every
weight from the softmax over the rows that a node sees.

Bounds: weights, relative 1e-4 of what is added plus 1e-6, as in
test_gpu_cache_loop.py (the lse's 1e-4 in every term); rows are copies.
"""
import glob
import math
import os
import re

import pytest
import torch

import cache_refs as ref
import exact_attention_48_gb300 as fa

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    with open(glob.glob(os.path.join(ROOT, "README*"))[0], encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "fa_fwd_tree" in b)


class Recorder:
    """The package, keeping what each call was given and returned."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args, **kw):
            held = [x.clone() if isinstance(x, torch.Tensor) else x for x in args]
            held_kw = {n: x.clone() if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
            out = getattr(fa, name)(*args, **kw)
            kept = tuple(x.clone() if isinstance(x, torch.Tensor) else x for x in out) if isinstance(out, tuple) \
                else out.clone() if isinstance(out, torch.Tensor) else out
            self.calls.append((name, held, held_kw, kept))
            return out
        return call

    def last(self, name):
        return [c for c in self.calls if c[0] == name][-1]


def true_weights(q, k, lens, parents, accepted, Nk):
    """What the accepted nodes' softmaxes give each row once the branch is the sequence's next rows: fp64 [B, Hkv, Nk];
    q, k as the tree call saw them, lens with all drafted rows counted."""
    B, H, Nt, d = q.shape
    Hkv = k.shape[1]
    w = torch.zeros(B, Hkv, Nk, dtype=torch.float64, device="cuda")
    for b in range(B):
        nodes = [x for x in accepted[b] if x >= 0]
        mask = ref.tree_mask(parents[b], lens[b], Nt, Nk).cuda()
        base = lens[b] - Nt
        for h in range(H):
            for node in nodes:
                rows = mask[node].nonzero()[:, 0]
                p = torch.softmax(q[b, h, node].double() @ k[b, h * Hkv // H, rows].double().T / math.sqrt(d), -1)
                at = torch.tensor([r if r < base else base + nodes.index(r - base) for r in rows.tolist()], device="cuda")
                w[b, h * Hkv // H, at] += p
    return w


@pytest.mark.parametrize("d", [64, 128])
def test_the_serving_step(d):
    g = ref.gen(600 + d)
    B, H, Hkv, N, Nk, Nt, keep = 3, 4, 2, 70, 110, 8, 72
    parents = [[-1, 0, 0, 1, 1, 2, 3, 5], [-1, 0, 1, 2, 0, 4, -2, -2], [-1, -1, 0, 1, 2, 3, 3, 6]]
    branches = [[[0, 2, 5, -1], [0, 1, 2, 3], [-1, -1, -1, -1]], [[0, 1, 3, 6], [-1, -1, -1, -1], [0, 2, 4, -1]]]
    kc, vc = (torch.full((B, Hkv, Nk, d), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kc[:, :, :N], vc[:, :, :N] = ref.draw(g, B, Hkv, N, d), ref.draw(g, B, Hkv, N, d)
    w = torch.zeros(B, Hkv, Nk, device="cuda")
    lens, code = ref.ints([N] * B), compile(example(), "example", "exec")
    names = {"torch": torch, "math": math, "d": d, "kc": kc, "vc": vc, "w": w, "keep": keep,
             "parents": ref.ints(parents)}
    depth = [[0] * Nt for _ in range(B)]
    for b in range(B):
        for i, p in enumerate(parents[b]):
            depth[b][i] = depth[b][p] + 1 if p >= 0 else 0
    truth, used = torch.zeros(B, Hkv, Nk, dtype=torch.float64, device="cuda"), [N] * B
    for step in range(2):
        q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nt, d), ref.draw(g, B, Hkv, Nt, d)
        k[1, :, 6:], v[1, :, 6:] = math.nan, math.inf          # padding nodes carry anything
        accepted = branches[step]
        rec = Recorder()
        names.update(fa=rec, q=q, k=k, v=v, lens=lens + Nt, positions=ref.ints(depth) + N + 4 * step,
                     accepted=ref.ints(accepted))
        exec(code, names)
        assert fa.fa_device_status() == 0
        # the weights
        _, (tq, tk, *_), _, _ = rec.last("fa_fwd_tree")
        add = true_weights(tq, tk, [n + Nt for n in used], parents, accepted, Nk)
        truth += add
        used = [n + sum(x >= 0 for x in accepted[b]) for b, n in enumerate(used)]
        got = rec.last("fa_key_weights")[3].double()
        for b, n in enumerate(used):
            err = (got[b, :, :n] - truth[b, :, :n]).abs()
            tol = 1e-4 * truth[b, :, :n] + 2.0 ** -22 * truth[b, :, :n] + 1e-6
            assert bool((err <= tol).all()), f"step {step} b{b}: {float(err.max()):.3e}"
            assert abs(float(add[b].sum()) - H * sum(x >= 0 for x in accepted[b])) <= 1e-9 * H * Nt
        # the cut: kept rows' keys and weights, and no weight behind them for the next rows to start from
        kept = rec.last("fa_cache_select")[3][0].tolist()
        lens = names["lens"]
        assert lens.tolist() == [min(n, keep) for n in used]
        before = rec.last("fa_cache_compact")[1]
        for b in range(B):
            for h in range(Hkv):
                rows = ref.select(rec.last("fa_key_weights")[3][b, h].cpu(), used[b], keep, 4, 64)
                assert kept[b][h] == rows, (step, b, h)
                at = torch.tensor([r for r in rows if r >= 0], device="cuda")
                assert torch.equal(kc[b, h, :len(at)], before[0][b, h, at])
                assert torch.equal(names["w"][b, h, :len(at)], rec.last("fa_key_weights")[3][b, h, at])
                assert not bool(names["w"][b, h, len(at):].any())
                truth[b, h] = torch.cat([truth[b, h, at], truth.new_zeros(Nk - len(at))])
        used = lens.tolist()
        assert bool(torch.isfinite(kc[:, :, :min(used)]).all())
