"""Cases of the operators around the key/value cache: rotary positions, attention
for a tree of drafted tokens, accumulated attention weight per key, eviction.

Each case runs in its plain form (elementary torch operations in fp32, angles in
64 bits) or, with ``own`` set, through the framework's calls on the same inputs.
"""
import math

import torch

own = False
DEV = "cuda"


def listed():
    return [
        # training step of the causal config (B4 H32 N4096 d128): q and k rotated before attention
        {"name": "rope_train_b4h32n4096", "op": "rope", "B": 4, "H": 32, "Hkv": 32, "N": 4096, "d": 128, "rot": 128,
         "interleaved": False, "bwd": False, "far": False, "layout": "bhnd"},
        # its backward with grouped heads, odd length, part of the head, long-context frequencies
        {"name": "rope_bwd_b8h16n2047", "op": "rope", "B": 8, "H": 16, "Hkv": 4, "N": 2047, "d": 64, "rot": 32,
         "interleaved": True, "bwd": True, "far": True, "layout": "bnhd"},
        # one new token per sequence, rotated and written to its cache rows before the decode call
        {"name": "append_step_b16h16", "op": "append", "B": 16, "H": 16, "Hkv": 16, "N": 1, "Nk": 4096, "d": 128,
         "rot": 128, "interleaved": False, "layout": "bhnd"},
        # a small draft against a short cache: latency
        {"name": "tree_b1h8t7nk1000", "op": "tree", "B": 1, "H": 8, "Hkv": 2, "Nt": 7, "Nk": 1000, "d": 64,
         "ragged": False, "layout": "bhnd"},
        # the decode workload's cache (B16 H16 Nk16384 d128), ragged lengths, 32 drafted tokens
        {"name": "tree_b16h16t32nk16384", "op": "tree", "B": 16, "H": 16, "Hkv": 16, "Nt": 32, "Nk": 16384, "d": 128,
         "ragged": True, "layout": "bhnd"},
        # long context, grouped heads, a wide draft, cache stored [B, Nk, H, d]
        {"name": "tree_b2h32kv8t64nk65536", "op": "tree", "B": 2, "H": 32, "Hkv": 8, "Nt": 64, "Nk": 65536, "d": 128,
         "ragged": False, "layout": "bnhd"},
        # a short window of queries added to the running sums
        {"name": "weights_b2h8q33nk1025", "op": "weights", "B": 2, "H": 8, "Hkv": 2, "Nq": 33, "Nk": 1025, "d": 64,
         "ragged": True, "causal": True, "add": True, "layout": "bhnd"},
        # every decode step: one query row against the decode workload's cache
        {"name": "weights_b16h16q1nk16384", "op": "weights", "B": 16, "H": 16, "Hkv": 16, "Nq": 1, "Nk": 16384,
         "d": 128, "ragged": False, "causal": True, "add": True, "layout": "bhnd"},
        # after the prompt: all queries of the causal config
        {"name": "weights_b4h32n4096", "op": "weights", "B": 4, "H": 32, "Hkv": 32, "Nq": 4096, "Nk": 4096, "d": 128,
         "ragged": False, "causal": True, "add": False, "layout": "bhnd"},
        # a small cache cut back: latency
        {"name": "evict_b1kv2nk640", "op": "evict", "B": 1, "Hkv": 2, "Nk": 640, "keep": 256, "d": 64, "first": 4,
         "recent": 32, "ragged": False, "layout": "bhnd"},
        # the decode workload's cache cut to half
        {"name": "evict_b16kv16nk16384", "op": "evict", "B": 16, "Hkv": 16, "Nk": 16384, "keep": 8192, "d": 128,
         "first": 4, "recent": 256, "ragged": False, "layout": "bhnd"},
        # one long sequence, few heads: long rows to select from
        {"name": "evict_b1kv8nk131072", "op": "evict", "B": 1, "Hkv": 8, "Nk": 131072, "keep": 16384, "d": 128,
         "first": 16, "recent": 1000, "ragged": True, "layout": "bnhd"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "tree", "tree", "weights", "weights", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 1, 2, 4, 8])
    B = _log(rng, 1, 16)
    layout = rng.choice(["bhnd", "bnhd"])
    if op == "rope":
        N = _log(rng, 1, min(16384, 4 * 32 * 4096 // (B * Hkv * G)))
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "N": N, "d": d, "rot": rng.choice([16, 32, d // 2, d]),
                "interleaved": rng.random() < 0.5, "bwd": rng.random() < 0.5, "far": rng.random() < 0.5,
                "layout": layout}
    if op == "append":
        Nk = _log(rng, 64, 4096)
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "N": _log(rng, 1, 64), "Nk": Nk, "d": d,
                "rot": rng.choice([16, 32, d // 2, d]), "interleaved": rng.random() < 0.5, "layout": layout}
    if op == "tree":
        Nt = _log(rng, 1, 128)
        cap = min(16 * 16 * 16384 // (B * Hkv), 2 * 32 * 64 * 65536 // (B * Hkv * G * Nt), 131072)
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "Nt": Nt, "Nk": _log(rng, min(Nt, cap), cap), "d": d,
                "ragged": rng.random() < 0.5, "layout": layout}
    if op == "weights":
        Nk = _log(rng, 1, min(65536, 16 * 16 * 16384 // (B * Hkv)))
        Nq = _log(rng, 1, max(1, min(Nk, 4096, 4 * 32 * 4096 * 2048 // (B * Hkv * G * Nk))))
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d,
                "ragged": rng.random() < 0.5, "causal": rng.random() < 0.7, "add": rng.random() < 0.5,
                "layout": layout}
    Nk = _log(rng, 64, min(131072, 16 * 16 * 16384 // (B * Hkv)))
    keep = max(1, int(Nk * rng.uniform(0.05, 0.5)))
    first = rng.randrange(0, keep // 4 + 1)
    return {"op": "evict", "B": B, "Hkv": Hkv, "Nk": Nk, "keep": keep, "d": d, "first": first,
            "recent": rng.randrange(0, keep - first + 1), "ragged": rng.random() < 0.5, "layout": layout}


def _lens(c, least):
    """Valid cache rows of each sequence: all, or between half and all of them."""
    B, Nk = c["B"], c["Nk"]
    return [max(min(Nk, least), Nk - (b * Nk) // (2 * B) if c["ragged"] else Nk) for b in range(B)]


def _frequencies(rot, far):
    """Angle per position of each pair; `far`: low frequencies slowed 16 times, as for a context 16 times as long."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    if far:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / 16.0 * (1.0 - keep)
    return f.float()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def rnd(B, H, N, layout="bhnd"):
        if layout == "bnhd":
            return torch.randn(B, N, H, c["d"], generator=g, device=DEV, dtype=torch.bfloat16).transpose(1, 2)
        return torch.randn(B, H, N, c["d"], generator=g, device=DEV, dtype=torch.bfloat16)

    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    s = {"case": c}
    if c["op"] == "rope":
        s["q"], s["k"] = rnd(B, c["H"], c["N"], c["layout"]), rnd(B, Hkv, c["N"], c["layout"])
        s["freq"] = _frequencies(c["rot"], c["far"])
        start = torch.randint(0, 1 << 20 if c["far"] else 64, (B, 1), generator=g, device=DEV, dtype=torch.int32)
        s["pos"] = start + torch.arange(c["N"], dtype=torch.int32, device=DEV)
        s["factor"] = 1.0 + 0.1 * math.log(16.0) if c["far"] else 1.0
        return s
    if c["op"] == "append":
        s["q"], s["k"], s["v"] = rnd(B, c["H"], c["N"]), rnd(B, Hkv, c["N"]), rnd(B, Hkv, c["N"])
        s["kc"], s["vc"] = rnd(B, Hkv, c["Nk"], c["layout"]), rnd(B, Hkv, c["Nk"], c["layout"])
        s["lens"] = torch.randint(min(c["N"], c["Nk"]), c["Nk"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["freq"] = _frequencies(c["rot"], False)
        return s
    if c["op"] == "tree":
        Nt = c["Nt"]
        s["q"] = rnd(B, c["H"], Nt)
        s["k"], s["v"] = rnd(B, Hkv, c["Nk"], c["layout"]), rnd(B, Hkv, c["Nk"], c["layout"])
        lens = _lens(c, Nt)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        i = torch.arange(Nt, device=DEV)
        u = torch.rand(B, Nt, generator=g, device=DEV) ** 0.5  # later nodes are likelier parents
        s["parents"] = (torch.minimum((u * (i + 1)).floor(), i.float()) - 1).to(torch.int32)
        if c["ragged"]:  # some drafts are shorter: their last nodes are padding
            used = torch.tensor([Nt - (5 * b) % (Nt // 4 + 1) for b in range(B)], device=DEV)
            s["parents"] = torch.where(i < used[:, None], s["parents"], torch.full_like(s["parents"], -2))
        return s
    if c["op"] == "weights":
        s["q"], s["k"] = rnd(B, c["H"], c["Nq"]), rnd(B, Hkv, c["Nk"], c["layout"])
        s["lens"] = torch.tensor(_lens(c, 1), dtype=torch.int32, device=DEV)
        s["lse"] = torch.logsumexp(_scores(s["q"], s["k"], _sees(c, s["lens"])), -1)
        s["w"] = torch.rand(B, Hkv, c["Nk"], generator=g, device=DEV) if c["add"] else None
        return s
    s["k"], s["v"] = rnd(B, Hkv, c["Nk"], c["layout"]), rnd(B, Hkv, c["Nk"], c["layout"])
    s["lens"] = torch.tensor(_lens(c, 1), dtype=torch.int32, device=DEV)
    w = torch.exp(2.0 * torch.randn(B, Hkv, c["Nk"], generator=g, device=DEV))
    # rows that no query has looked at weigh nothing, and some weights are alike
    s["w"] = torch.where(w < 0.08, torch.zeros_like(w), torch.where(w < 0.3, torch.full_like(w, 0.25), w))
    s["k_out"], s["v_out"] = (torch.zeros(B, Hkv, c["keep"], d, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    s["w_out"] = torch.zeros(B, Hkv, c["keep"], device=DEV)
    return s


# ---------------------------------------------------------------- plain forms


def _sees(c, lens):
    """[B, Nq, Nk]: the query rows are the last Nq positions of each sequence."""
    j = torch.arange(c["Nk"], device=DEV)
    i = torch.arange(c["Nq"], device=DEV)
    last = lens[:, None] - c["Nq"] + i if c["causal"] else (lens - 1)[:, None].expand(-1, c["Nq"])
    return j <= torch.minimum(last, lens[:, None] - 1)[:, :, None]


def _scores(q, k, sees):
    """[B, H, Nq, Nk] scaled scores, -inf where hidden."""
    B, H, Nq, d = q.shape
    Hkv = k.shape[1]
    s = torch.matmul(q.float().reshape(B, Hkv, -1, d), k.float().transpose(-1, -2)) * (1.0 / math.sqrt(d))
    return s.view(B, H, Nq, -1).masked_fill_(~sees[:, None], -math.inf)


def _rotate(x, cos, sin, rot, interleaved):
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, y[..., rot:]), -1).to(torch.bfloat16)


def _turn(pos, freq, factor, sign):
    """cos and sin [B, 1, N, rot/2] of the positions' angles, times the factor."""
    ang = pos.double()[:, None, :, None] * freq.double()
    return (ang.cos() * factor).float(), (ang.sin() * (factor * sign)).float()


def _sees_tree(parents, lens, Nk):
    """[B, Nt, Nk]: the rows before the tree, the node's own row and its ancestors' rows; nothing for padding."""
    B, Nt = parents.shape
    i = torch.arange(Nt, device=DEV)
    base = (lens - Nt).long()
    dead = (parents < -1) | (parents >= i) | (base[:, None] + i < 0)
    reach = torch.eye(Nt, device=DEV) + (parents[:, :, None] == i).float()
    for _ in range(max(1, (Nt - 1).bit_length())):
        reach = (reach @ reach).clamp_(max=1.0)
    dead = (reach @ dead.float()[:, :, None])[..., 0] > 0
    j = torch.arange(Nk, device=DEV)
    node = j - base[:, None]  # [B, Nk]
    inside = (node >= 0) & (node < Nt)
    up = torch.gather(reach, 2, node.clamp(0, Nt - 1)[:, None, :].expand(-1, Nt, -1)) > 0
    return ((node < 0)[:, None] | (inside[:, None] & up)) & ~dead[:, :, None]


def _keep(w, lens, keep, first, recent):
    """kept [B, H, keep] int32 ascending (-1 behind a short sequence's rows) and the new lengths."""
    Nk = w.shape[-1]
    j = torch.arange(Nk, device=DEV)
    n = lens.long()[:, None, None]
    must = (j < first) | (j >= n - recent)
    score = torch.where(j < n, torch.where(must, torch.full_like(w, math.inf), w), torch.full_like(w, -math.inf))
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :keep]
    kept = torch.sort(torch.where(order < n, order, torch.full_like(order, Nk)), dim=-1)[0]
    return torch.where(kept < Nk, kept, torch.full_like(kept, -1)).to(torch.int32), lens.clamp(max=keep)


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "rope":
        cos, sin = _turn(state["pos"], state["freq"], state["factor"], -1.0 if c["bwd"] else 1.0)
        return [_rotate(x, cos, sin, c["rot"], c["interleaved"]) for x in (state["q"], state["k"])]
    if c["op"] == "append":
        rows = state["lens"][:, None] - c["N"] + torch.arange(c["N"], dtype=torch.int32, device=DEV)
        cos, sin = _turn(rows, state["freq"], 1.0, 1.0)
        b, r = torch.nonzero(rows >= 0, as_tuple=True)
        at = rows[b, r].long()
        state["kc"][b, :, at] = _rotate(state["k"], cos, sin, c["rot"], c["interleaved"])[b, :, r]
        state["vc"][b, :, at] = state["v"][b, :, r]
        return [_rotate(state["q"], cos, sin, c["rot"], c["interleaved"]), state["kc"], state["vc"]]
    if c["op"] == "tree":
        q, v = state["q"], state["v"]
        s = _scores(q, state["k"], _sees_tree(state["parents"], state["lens"], c["Nk"]))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(c["B"], c["Hkv"], -1, c["Nk"]), v.float()).view(q.shape)
        o = torch.where(l > 0, o / l, torch.zeros_like(o))
        return [o.to(torch.bfloat16), (m + torch.log(l))[..., 0]]
    if c["op"] == "weights":
        p = torch.exp(_scores(state["q"], state["k"], _sees(c, state["lens"])) - state["lse"].masked_fill(
            state["lse"] == -math.inf, 0.0)[..., None])
        w = p.view(c["B"], c["Hkv"], -1, c["Nk"]).sum(2)
        return [w if state["w"] is None else state["w"] + w]
    kept, lens = _keep(state["w"], state["lens"], c["keep"], c["first"], c["recent"])
    at, on = kept.clamp(min=0).long(), kept >= 0
    for x, y in (("k", "k_out"), ("v", "v_out")):
        rows = torch.gather(state[x], 2, at[..., None].expand(-1, -1, -1, c["d"]))
        state[y].copy_(torch.where(on[..., None], rows, state[y]))
    state["w_out"].copy_(torch.where(on, torch.gather(state["w"], 2, at), state["w_out"]))
    return [kept, lens, state["k_out"], state["v_out"], state["w_out"]]


def _own(c, s):
    import exact_attention_48_gb300 as fa

    if c["op"] == "rope":
        call = fa.fa_rope_bwd if c["bwd"] else fa.fa_rope
        return list(call(s["q"], s["k"], s["freq"], s["pos"], interleaved=c["interleaved"], factor=s["factor"]))
    if c["op"] == "append":
        q = fa.fa_rope_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["lens"], s["freq"],
                              interleaved=c["interleaved"])
        return [q, s["kc"], s["vc"]]
    if c["op"] == "tree":
        return list(fa.fa_fwd_tree(s["q"], s["k"], s["v"], s["parents"], s["lens"]))
    if c["op"] == "weights":
        return [fa.fa_key_weights(s["q"], s["k"], s["lse"], s["lens"], causal=c["causal"], weights_in=s["w"])]
    kept, lens = fa.fa_cache_select(s["w"], c["keep"], s["lens"], first=c["first"], recent=c["recent"])
    fa.fa_cache_compact(s["k"], s["v"], kept, weights=s["w"], k_out=s["k_out"], v_out=s["v_out"],
                        weights_out=s["w_out"])
    return [kept, lens, s["k_out"], s["v_out"], s["w_out"]]


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "rope":
        rows = B * (c["H"] + Hkv) * c["N"]
        return {"bytes": 4 * rows * d + 4 * B * c["N"], "flops": 3 * rows * c["rot"]}
    if c["op"] == "append":
        rows = B * c["N"]
        return {"bytes": 4 * rows * (c["H"] + 2 * Hkv) * d, "flops": 3 * rows * (c["H"] + Hkv) * c["rot"]}
    if c["op"] == "tree":
        n, rows = sum(_lens(c, c["Nt"])), B * c["H"] * c["Nt"]
        return {"bytes": 4 * Hkv * n * d + rows * (4 * d + 4), "flops": 4 * c["H"] * c["Nt"] * n * d}
    if c["op"] == "weights":
        n, Nq = _lens(c, 1), c["Nq"]
        pairs = sum(_pairs(x, Nq, c["causal"]) for x in n)
        return {"bytes": 2 * Hkv * sum(n) * d + B * c["H"] * Nq * (2 * d + 4) + B * Hkv * c["Nk"] * (8 if c["add"] else 4),
                "flops": 2 * c["H"] * pairs * d}
    kept = sum(min(c["keep"], x) for x in _lens(c, 1))
    return {"bytes": Hkv * (4 * sum(_lens(c, 1)) + kept * (8 * d + 8) + 4 * B * c["keep"]), "flops": 0}


def _pairs(n, Nq, causal):
    """(query, key) pairs that the mask leaves."""
    if not causal:
        return n * Nq
    first = max(0, n - Nq + 1)  # keys that the first query row with any sees
    return (first + n) * (n - first + 1) // 2


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("rope", "append"):
        if c["op"] == "rope":
            pos, factor, sign = s["pos"].double(), s["factor"], (-1.0 if c["bwd"] else 1.0)
        else:
            pos = (s["lens"].double()[:, None] - c["N"]) + torch.arange(c["N"], dtype=torch.float64, device=DEV)
            factor, sign = 1.0, 1.0
        turn = torch.polar(torch.full_like(pos, factor)[..., None].expand(-1, -1, c["rot"] // 2).contiguous(),
                           sign * pos[..., None] * s["freq"].double())[:, None]

        def one(x):
            x = x.double().clone()
            if c["interleaved"]:
                z = torch.view_as_complex(x[..., :c["rot"]].reshape(*x.shape[:-1], -1, 2).contiguous()) * turn
                x[..., :c["rot"]] = torch.view_as_real(z).flatten(-2)
            else:
                h = c["rot"] // 2
                z = torch.complex(x[..., :h].contiguous(), x[..., h:c["rot"]].contiguous()) * turn
                x[..., :h], x[..., h:c["rot"]] = z.real, z.imag
            return x

        if c["op"] == "rope":
            return [one(s["q"]), one(s["k"])]
        q, k, kc, vc = one(s["q"]), one(s["k"]), s["kc"].double(), s["vc"].double()
        for b, n in enumerate(s["lens"].tolist()):
            for i in range(c["N"]):
                if 0 <= n - c["N"] + i:
                    kc[b, :, n - c["N"] + i], vc[b, :, n - c["N"] + i] = k[b, :, i], s["v"][b, :, i].double()
        return [q, kc, vc]
    if c["op"] == "tree":
        Nt, G = c["Nt"], c["H"] // c["Hkv"]
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
        for b, (n, parents) in enumerate(zip(s["lens"].tolist(), s["parents"].tolist())):
            sees, lives = [], []
            for i, p in enumerate(parents):  # what a node sees of the tree: what its parent sees, and itself
                lives.append(-1 <= p < i and n - Nt + i >= 0 and (p < 0 or lives[p]))
                sees.append((sees[p] if lives[i] and p >= 0 else frozenset()) | {i})
            mask = torch.zeros(Nt, n, dtype=torch.bool)
            for i in range(Nt):
                if lives[i]:
                    mask[i, :max(0, n - Nt)] = True
                    mask[i, [n - Nt + x for x in sees[i]]] = True
            live = torch.tensor(lives, device=DEV)
            mask = mask.to(DEV)
            for h in range(c["Hkv"]):
                k, v = s["k"][b, h, :n].double(), s["v"][b, h, :n].double()
                for hq in range(h * G, h * G + G):
                    t = (s["q"][b, hq].double() @ k.T / math.sqrt(c["d"])).masked_fill(~mask, -math.inf)[live]
                    lse[b, hq, live] = torch.logsumexp(t, -1)
                    o[b, hq, live] = torch.softmax(t, -1) @ v
        return [o, lse]
    if c["op"] == "weights":
        G, Nq = c["H"] // c["Hkv"], c["Nq"]
        w = torch.zeros(c["B"], c["Hkv"], c["Nk"], dtype=torch.float64, device=DEV)
        if s["w"] is not None:
            w += s["w"].double()
        i = torch.arange(Nq, device=DEV)[:, None]
        for b, n in enumerate(s["lens"].tolist()):
            hide = torch.arange(n, device=DEV) > n - Nq + i
            for h in range(c["H"]):
                t = s["q"][b, h].double() @ s["k"][b, h // G, :n].double().T / math.sqrt(c["d"])
                p = torch.exp(t - s["lse"][b, h].double().clamp(min=-1e300)[:, None])
                w[b, h // G, :n] += (p.masked_fill_(hide, 0.0) if c["causal"] else p).sum(0)
        return [w]
    lens = s["lens"].tolist()
    w = s["w"].cpu().numpy()
    out = [torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in (s["k_out"], s["v_out"], s["w_out"])]
    for b, n in enumerate(lens):
        for h in range(c["Hkv"]):
            rows = list(range(n))
            if n > c["keep"]:
                a, z = c["first"], n - c["recent"]
                by = w[b, h, a:z].argsort(kind="stable")  # ascending: the last ones, ties by hand
                need = c["keep"] - a - c["recent"]
                middle = []
                if need:
                    edge = w[b, h, a + by[len(by) - need]]
                    over = [a + x for x in (w[b, h, a:z] > edge).nonzero()[0]]
                    ties = [a + x for x in (w[b, h, a:z] == edge).nonzero()[0]]
                    middle = sorted(over + ties[:need - len(over)])
                rows = list(range(a)) + middle + list(range(z, n))
            at = torch.tensor([int(x) for x in rows], dtype=torch.int64, device=DEV)
            out[0][b, h, :len(rows)] = s["k"][b, h, at].double()
            out[1][b, h, :len(rows)] = s["v"][b, h, at].double()
            out[2][b, h, :len(rows)] = s["w"][b, h, at].double()
    return [None, None] + out
