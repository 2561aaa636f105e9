"""Cases of serving from a key/value cache held in 8 bits: the append of new rows, attention of the newest rows or
of a drafted tree, rows moved together, and the verification of drafted tokens.

A cache holds e4m3 codes and, for each block of rows of a head, one power of two by which they are scaled. Each case
runs in its plain form (elementary torch operations in fp32; angles, sums over a vocabulary and what is compared with
them in 64 bits) or, with ``own`` set, through the framework's calls on the same inputs.
"""
import math

import torch

own = False
DEV = "cuda"


def listed():
    return [
        # one new token per sequence of the decode workload (B16 H16 d128)
        {"name": "append_step_b16h16", "op": "append", "B": 16, "H": 16, "Hkv": 16, "N": 1, "Nk": 4096, "d": 128,
         "rot": 128, "interleaved": False, "block": 64, "layout": "bhnd"},
        # a prompt of odd length, grouped heads, cache stored [B, Nk, H, d]
        {"name": "append_b4h32kv8n4001", "op": "append", "B": 4, "H": 32, "Hkv": 8, "N": 4001, "Nk": 8192, "d": 128,
         "rot": 64, "interleaved": True, "block": 128, "layout": "bnhd"},
        # one query row against a short cache: latency
        {"name": "attend_b1h8t1nk1000", "op": "attend", "B": 1, "H": 8, "Hkv": 2, "Nt": 1, "Nk": 1000, "d": 64,
         "block": 64, "tree": False, "ragged": False, "layout": "bhnd"},
        # the decode workload's cache (B16 H16 Nk16384 d128), one token each
        {"name": "attend_b16h16t1nk16384", "op": "attend", "B": 16, "H": 16, "Hkv": 16, "Nt": 1, "Nk": 16384, "d": 128,
         "block": 64, "tree": False, "ragged": False, "layout": "bhnd"},
        # long contexts, grouped heads, a chain of drafted tokens, cache stored [B, Nk, H, d]
        {"name": "attend_b2h32kv8t5nk100001", "op": "attend", "B": 2, "H": 32, "Hkv": 8, "Nt": 5, "Nk": 100001,
         "d": 128, "block": 32, "tree": False, "ragged": False, "layout": "bnhd"},
        # the decode workload's cache, ragged lengths, a tree of 32 drafted tokens
        {"name": "attend_b16h16t32nk16384", "op": "attend", "B": 16, "H": 16, "Hkv": 16, "Nt": 32, "Nk": 16384,
         "d": 128, "block": 64, "tree": True, "ragged": True, "layout": "bhnd"},
        # a wide tree over long contexts, grouped heads
        {"name": "attend_b2h32kv8t64nk65536", "op": "attend", "B": 2, "H": 32, "Hkv": 8, "Nt": 64, "Nk": 65536,
         "d": 128, "block": 128, "tree": True, "ragged": False, "layout": "bhnd"},
        # a small cache cut back: latency
        {"name": "evict_b1kv2nk640", "op": "evict", "B": 1, "Hkv": 2, "Nk": 640, "keep": 257, "d": 64, "block": 16,
         "layout": "bhnd"},
        # the decode workload's cache cut to half
        {"name": "evict_b16kv16nk16384", "op": "evict", "B": 16, "Hkv": 16, "Nk": 16384, "keep": 8192, "d": 128,
         "block": 64, "layout": "bhnd"},
        # a chain of drafted tokens of one sequence: latency
        {"name": "verify_b1t5v32000", "op": "verify", "B": 1, "Nt": 5, "V": 32000, "tree": False, "draft": True},
        # a batch of short chains, odd vocabulary, drafted without probabilities
        {"name": "verify_b64t8v50021", "op": "verify", "B": 64, "Nt": 8, "V": 50021, "tree": True, "draft": False},
        # a batch of trees, large vocabulary
        {"name": "verify_b16t32v131072", "op": "verify", "B": 16, "Nt": 32, "V": 131072, "tree": True, "draft": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "evict", "verify", "verify"])
    if op == "verify":
        B = _log(rng, 1, 64)
        V = _log(rng, 1000, 131072)
        Nt = _log(rng, 1, max(1, min(64, 16 * 32 * 131072 // (B * V))))
        return {"op": op, "B": B, "Nt": Nt, "V": V, "tree": rng.random() < 0.6, "draft": rng.random() < 0.7}
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 1, 2, 4, 8])
    B = _log(rng, 1, 16)
    block = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["bhnd", "bnhd"])
    if op == "append":
        N = 1 if rng.random() < 0.3 else _log(rng, 1, min(4096, 4 * 48 * 4001 // (B * Hkv * (G + 2))))
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "N": N, "Nk": _log(rng, max(64, N), 8192), "d": d,
                "rot": rng.choice([16, 32, d // 2, d]), "interleaved": rng.random() < 0.5, "block": block,
                "layout": layout}
    if op == "attend":
        Nt = 1 if rng.random() < 0.4 else _log(rng, 1, 128)
        cap = min(16 * 16 * 16384 // (B * Hkv), 2 * 32 * 64 * 65536 // (B * Hkv * G * Nt), 131072)
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "Nt": Nt, "Nk": _log(rng, min(Nt, cap), cap), "d": d,
                "block": block, "tree": rng.random() < 0.5, "ragged": rng.random() < 0.5, "layout": layout}
    Nk = _log(rng, 64, min(131072, 16 * 16 * 16384 // (B * Hkv)))
    return {"op": op, "B": B, "Hkv": Hkv, "Nk": Nk, "keep": max(1, int(Nk * rng.uniform(0.05, 0.5))), "d": d,
            "block": block, "layout": layout}


def _lens(c, least):
    """Valid cache rows of each sequence: all, or between half and all of them."""
    B, Nk = c["B"], c["Nk"]
    return [max(min(Nk, least), Nk - (b * Nk) // (2 * B) if c["ragged"] else Nk) for b in range(B)]


def _blocks(c, rows):
    return (rows + c["block"] - 1) // c["block"]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    B = c["B"]
    if c["op"] == "verify":
        return _prepare_verify(c, s, g)

    def rnd(H, N, layout="bhnd"):
        if layout == "bnhd":
            return torch.randn(B, N, H, c["d"], generator=g, device=DEV, dtype=torch.bfloat16).transpose(1, 2)
        return torch.randn(B, H, N, c["d"], generator=g, device=DEV, dtype=torch.bfloat16)

    def cache():
        """Codes [B, Hkv, Nk, d] and scales [B, Hkv, blocks] of random rows."""
        Hkv, Nk, d, nb = c["Hkv"], c["Nk"], c["d"], _blocks(c, c["Nk"])
        shape = (B, Nk, Hkv, d) if c["layout"] == "bnhd" else (B, Hkv, Nk, d)
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
        codes = codes.transpose(1, 2) if c["layout"] == "bnhd" else codes
        scale = torch.empty(B, Hkv, nb, device=DEV)
        for b in range(B):  # (a sequence at a time: little memory beside the codes)
            x = torch.zeros(Hkv, nb * c["block"], d, device=DEV)
            x[:, :Nk] = torch.randn(Hkv, Nk, d, generator=g, device=DEV)
            x = x.view(Hkv, nb, -1)
            scale[b] = _least_scale(x.abs().amax(-1))
            codes[b] = (x / scale[b][..., None]).view(Hkv, -1, d)[:, :Nk].to(torch.float8_e4m3fn)
        return codes, scale

    s["kc"], s["ks"] = cache()
    s["vc"], s["vs"] = cache()
    if c["op"] == "append":
        s["q"], s["k"], s["v"] = rnd(c["H"], c["N"]), rnd(c["Hkv"], c["N"]), rnd(c["Hkv"], c["N"])
        s["lens"] = torch.randint(c["N"], c["Nk"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])).float()
        return s
    if c["op"] == "attend":
        Nt = c["Nt"]
        s["q"] = rnd(c["H"], Nt)
        s["lens"] = torch.tensor(_lens(c, Nt), dtype=torch.int32, device=DEV)
        s["parents"] = _random_tree(B, Nt, g) if c["tree"] else None
        if c["tree"] and c["ragged"]:  # some drafts are shorter: their last nodes are padding
            i = torch.arange(Nt, device=DEV)
            used = torch.tensor([Nt - (5 * b) % (Nt // 4 + 1) for b in range(B)], device=DEV)
            s["parents"] = torch.where(i < used[:, None], s["parents"], torch.full_like(s["parents"], -2))
        return s
    # the rows of each head that are kept: any `keep` of them, ascending
    order = torch.rand(B, c["Hkv"], c["Nk"], generator=g, device=DEV).argsort(-1)[..., :c["keep"]]
    s["kept"] = order.sort(-1)[0].to(torch.int32)
    shape = (B, c["Hkv"], c["keep"], c["d"])
    s["ko"], s["vo"] = (torch.zeros(shape, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    s["kso"], s["vso"] = (torch.zeros(B, c["Hkv"], _blocks(c, c["keep"]), device=DEV) for _ in range(2))
    return s


def _random_tree(B, Nt, g):
    """Node 0 follows the rows before the tree; later nodes are likelier parents."""
    i = torch.arange(Nt, device=DEV)
    u = torch.rand(B, Nt, generator=g, device=DEV) ** 0.5
    parents = torch.minimum((u * i).floor(), (i - 1).float()).to(torch.int32)
    parents[:, 0] = -1
    return parents


def _prepare_verify(c, s, g):
    B, Nt, V = c["B"], c["Nt"], c["V"]
    if c["tree"]:
        parents = _random_tree(B, Nt, g)
    else:
        parents = (torch.arange(Nt, device=DEV, dtype=torch.int32) - 1).expand(B, Nt).contiguous()
    up = parents.clamp(min=0).long()
    logits = 3.0 * torch.randn(B, Nt, V, generator=g, device=DEV)
    s["p"] = torch.softmax(logits, -1)
    if c["draft"]:  # a draft model that is near the target
        logits.mul_(0.9).add_(torch.randn(B, Nt, V, generator=g, device=DEV), alpha=0.8)
        s["q"] = torch.softmax(logits, -1)
        del logits
        from_row = torch.gather(s["q"].cumsum(-1, dtype=torch.float64), 1, up[..., None].expand(-1, -1, V))
        u = torch.rand(B, Nt, 1, generator=g, device=DEV, dtype=torch.float64) * from_row[..., -1:]
        tokens = torch.searchsorted(from_row, u, right=True)[..., 0].clamp(max=V - 1)
    else:  # the likeliest tokens, the nth child of a node the nth of them
        s["q"] = None
        i = torch.arange(Nt, device=DEV)
        rank = ((parents[:, None, :] == parents[:, :, None]) & (i[None, :] < i[:, None])).sum(-1)
        best = logits.topk(min(V, 8), -1)[1]
        tokens = torch.gather(best, 1, up[..., None].expand(-1, -1, best.shape[-1]))
        tokens = torch.gather(tokens, 2, rank.clamp(max=best.shape[-1] - 1)[..., None])[..., 0]
    s["parents"], s["tokens"] = parents, tokens.to(torch.int32)
    s["u"] = torch.rand(B, Nt, generator=g, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms


def _least_scale(a):
    """The least power of two, 2^-100 or more, by which values of up to `a` fit e4m3 (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(a)
    return torch.ldexp(torch.ones_like(a), (e - 9 + (m > 0.875).int()).clamp(min=-100))


def _values(codes, scale, block):
    """The fp32 values [B, Hkv, Nk, d] that a cache stands for."""
    return codes.float() * scale.repeat_interleave(block, -1)[..., :codes.shape[2], None]


def _rotate(x, cos, sin, rot, interleaved):
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _append(c, x, lens, codes, scale):
    """Rows x [B, Hkv, N, d] (fp32) become the last N of each sequence's rows, in place."""
    B, Hkv, N, d = x.shape
    Nk, block, nb = c["Nk"], c["block"], scale.shape[-1]
    start = (lens.long() - N)[:, None]                                       # rows before the new ones
    rows = start + torch.arange(N, device=DEV)
    at = (rows // block)[:, None].expand(-1, Hkv, -1)
    most = torch.zeros(B, Hkv, nb, device=DEV).scatter_reduce_(2, at, x.abs().amax(-1), "amax")
    first = torch.arange(nb, device=DEV) * block
    new = ((first + block > start) & (first < lens[:, None]))[:, None]       # blocks with new rows
    held = torch.where((first < start)[:, None], scale, torch.zeros_like(scale))
    now = torch.where(new, torch.maximum(held, _least_scale(most)), scale)
    # the rows of the block that is continued, in its new scale
    b, r = torch.nonzero(torch.arange(block, device=DEV) < start % block, as_tuple=True)
    old = (start[b, 0] // block) * block + r
    blk = start[b, 0] // block
    raw = codes.view(torch.uint8)
    keep = raw[b, :, old].view(torch.float8_e4m3fn).float() * (scale[b, :, blk] / now[b, :, blk])[..., None]
    grown = now[b, :, blk] > scale[b, :, blk]
    raw[b, :, old] = torch.where(grown[..., None], keep.to(torch.float8_e4m3fn).view(torch.uint8), raw[b, :, old])
    y = (x / torch.gather(now, 2, at)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    raw[torch.arange(B, device=DEV)[:, None], :, rows] = y.transpose(1, 2)
    scale.copy_(now)


def _sees(c, parents, lens):
    """[B, Nt, Nk]: the rows before the tree, the node's own row and its ancestors' rows; nothing for padding."""
    B, Nt, Nk = c["B"], c["Nt"], c["Nk"]
    i = torch.arange(Nt, device=DEV)
    base = (lens - Nt).long()
    if parents is None:
        parents = (i - 1).expand(B, Nt)
    dead = (parents < -1) | (parents >= i) | (base[:, None] + i < 0)
    reach = torch.eye(Nt, device=DEV) + (parents[:, :, None] == i).float()
    for _ in range(max(1, (Nt - 1).bit_length())):
        reach = (reach @ reach).clamp_(max=1.0)
    dead = (reach @ dead.float()[:, :, None])[..., 0] > 0
    node = torch.arange(Nk, device=DEV) - base[:, None]
    inside = (node >= 0) & (node < Nt)
    up = torch.gather(reach, 2, node.clamp(0, Nt - 1)[:, None, :].expand(-1, Nt, -1)) > 0
    return ((node < 0)[:, None] | (inside[:, None] & up)) & ~dead[:, :, None]


def _attend(c, s):
    q, k = s["q"], _values(s["kc"], s["ks"], c["block"])
    B, H, Nt, d = q.shape
    t = torch.matmul(q.float().reshape(B, c["Hkv"], -1, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    t = t.view(B, H, Nt, -1).masked_fill_(~_sees(c, s["parents"], s["lens"])[:, None], -math.inf)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, c["Hkv"], -1, c["Nk"]), _values(s["vc"], s["vs"], c["block"])).view(q.shape)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return [o.to(torch.bfloat16), (m + torch.log(l))[..., 0]]


def _move(c, kept, codes, scale, codes_out, scale_out):
    """Rows `kept` of each head, every block in the greatest scale of the blocks its rows come from."""
    B, Hkv, M = kept.shape
    block = c["block"]
    rows = kept.long()
    of = torch.gather(scale, 2, rows // block)                               # [B, Hkv, M]
    to = (torch.arange(M, device=DEV) // block).expand(B, Hkv, M)
    now = torch.zeros_like(scale_out).scatter_reduce_(2, to, of, "amax")
    y = torch.gather(codes.view(torch.uint8), 2, rows[..., None].expand(-1, -1, -1, c["d"]))
    y = y.view(torch.float8_e4m3fn).float() * (of / torch.gather(now, 2, to))[..., None]
    codes_out.copy_(y.to(torch.float8_e4m3fn))
    scale_out.copy_(now)


def _verify(c, s):
    """The nodes accepted, in order; how many; the token that follows them."""
    B, Nt, V = c["B"], c["Nt"], c["V"]
    parents, tokens = s["parents"], s["tokens"].long()
    seq = torch.arange(B, device=DEV)
    node = torch.zeros(B, dtype=torch.long, device=DEV)
    accepted = torch.full((B, Nt), -1, dtype=torch.int32, device=DEV)
    accepted[:, 0] = 0
    count = torch.ones(B, dtype=torch.long, device=DEV)
    rest = s["p"][:, 0].double()                                             # what children have left of p
    total = torch.ones(B, dtype=torch.float64, device=DEV)
    for i in range(1, Nt):  # a node's children come after it
        x = tokens[:, i]
        asked = parents[:, i] == node
        if s["q"] is None:
            q = (torch.arange(V, device=DEV) == x[:, None]).double()
        else:
            q = s["q"][seq, node].double()
        yes = asked & (s["u"][:, i].double() * q[seq, x] * total < rest[seq, x])
        no = asked & ~yes
        less = (rest - total[:, None] * q).clamp(min=0.0)
        rest = torch.where(yes[:, None], s["p"][:, i].double(), torch.where(no[:, None], less, rest))
        total = torch.where(yes, torch.ones_like(total), torch.where(no, rest.sum(-1), total))
        node = torch.where(yes, torch.full_like(node, i), node)
        accepted[seq, count.clamp(max=Nt - 1)] = torch.where(yes, node.int(), accepted[seq, count.clamp(max=Nt - 1)])
        count = count + yes.long()
    rest = torch.where(rest.sum(-1, keepdim=True) > 0.0, rest, s["p"][seq, node].double())
    below = rest.cumsum(-1)
    token = (below <= s["u"][:, :1].double() * below[:, -1:]).sum(-1)
    return [accepted, count.int(), token.int()]


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "append":
        pos = (state["lens"][:, None] - c["N"] + torch.arange(c["N"], device=DEV)).double()
        ang = pos[:, None, :, None] * state["freq"].double()
        cos, sin = ang.cos().float(), ang.sin().float()
        q = _rotate(state["q"], cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)
        _append(c, _rotate(state["k"], cos, sin, c["rot"], c["interleaved"]), state["lens"], state["kc"], state["ks"])
        _append(c, state["v"].float(), state["lens"], state["vc"], state["vs"])
        return [q, state["kc"], state["ks"], state["vc"], state["vs"]]
    if c["op"] == "attend":
        return _attend(c, state)
    if c["op"] == "evict":
        _move(c, state["kept"], state["kc"], state["ks"], state["ko"], state["kso"])
        _move(c, state["kept"], state["vc"], state["vs"], state["vo"], state["vso"])
        return [state["ko"], state["kso"], state["vo"], state["vso"]]
    return _verify(c, state)


def _own(c, s):
    import exact_attention_48_gb300 as fa

    if c["op"] == "append":
        q = fa.fa_rope_append_fp8(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["lens"], s["freq"],
                                  interleaved=c["interleaved"], block=c["block"])
        return [q, s["kc"], s["ks"], s["vc"], s["vs"]]
    if c["op"] == "attend":
        return list(fa.fa_fwd_tree_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["parents"], s["lens"],
                                       block=c["block"]))
    if c["op"] == "evict":
        fa.fa_cache_compact_fp8(s["kc"], s["vc"], s["ks"], s["vs"], s["kept"], block=c["block"], k_out=s["ko"],
                                v_out=s["vo"], k_scale_out=s["kso"], v_scale_out=s["vso"])
        return [s["ko"], s["kso"], s["vo"], s["vso"]]
    return list(fa.fa_tree_verify(s["parents"], s["tokens"], s["p"], s["q"], s["u"]))


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "verify":  # a row of the target, and of the draft, for the token that follows
        rows = c["B"] * (2 if c["draft"] else 1)
        return {"bytes": 4 * rows * c["V"] + 24 * c["B"] * c["Nt"], "flops": 3 * c["B"] * c["V"]}
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "append":
        tokens = B * c["N"]
        return {"bytes": tokens * d * (4 * c["H"] + 6 * Hkv) + 8 * Hkv * B * _blocks(c, c["N"]),
                "flops": 3 * tokens * (c["H"] + Hkv) * c["rot"] + 2 * tokens * 2 * Hkv * d}
    if c["op"] == "attend":
        n, rows = sum(_lens(c, c["Nt"])), B * c["H"] * c["Nt"]
        return {"bytes": 2 * Hkv * n * d + 8 * Hkv * n // c["block"] + rows * (4 * d + 4),
                "flops": 4 * c["H"] * c["Nt"] * n * d}
    kept = B * Hkv * c["keep"]
    return {"bytes": kept * (4 * d + 4) + 8 * B * Hkv * (_blocks(c, c["Nk"]) + _blocks(c, c["keep"])), "flops": 0}


# ---------------------------------------------------------------- 64 bits


def _to_e4m3(x):
    """Reals of up to 448 in size to the nearest values of e4m3 (steps of 2^-3 of the leading power, 2^-9 at least; ties to even)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _fitting(a):
    """2^ceil(log2(a / 448)), 2^-100 or more."""
    e = torch.ceil(torch.log2((a / 448.0).clamp(min=2.0 ** -100)))
    return torch.exp2(e)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "append":
        lens, rot, N, block = s["lens"].tolist(), c["rot"], c["N"], c["block"]
        pos = (s["lens"].double()[:, None] - N) + torch.arange(N, dtype=torch.float64, device=DEV)
        a = pos[..., None] * s["freq"].double()
        turn = torch.polar(torch.ones_like(a), a)[:, None]

        def turned(x):
            x = x.double().clone()
            if c["interleaved"]:
                z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], -1, 2).contiguous()) * turn
                x[..., :rot] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
                x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
            return x

        def append(x, codes, scale):
            codes, scale = codes.double(), scale.double()
            for b, n in enumerate(lens):
                for blk in range((n - N) // block, (n - 1) // block + 1):
                    lo, hi = max(n - N, blk * block), min(n, (blk + 1) * block)
                    part = x[b, :, lo - (n - N):hi - (n - N)]
                    now = _fitting(part.abs().amax((1, 2)))
                    if lo > blk * block:
                        was = scale[b, :, blk]
                        now = torch.maximum(now, was)
                        old = codes[b, :, blk * block:lo]
                        codes[b, :, blk * block:lo] = _to_e4m3(old * (was / now)[:, None, None])
                    codes[b, :, lo:hi] = _to_e4m3(part / now[:, None, None])
                    scale[b, :, blk] = now
            return codes, scale

        return [turned(s["q"]), *append(turned(s["k"]), s["kc"], s["ks"]), *append(s["v"].double(), s["vc"], s["vs"])]
    if c["op"] == "attend":
        Nt, G = c["Nt"], c["H"] // c["Hkv"]
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
        trees = [list(range(-1, Nt - 1))] * c["B"] if s["parents"] is None else s["parents"].tolist()
        for b, (n, parents) in enumerate(zip(s["lens"].tolist(), trees)):
            sees, lives = [], []
            for i, p in enumerate(parents):  # what a node sees of the tree: what its parent sees, and itself
                lives.append(-1 <= p < i and n - Nt + i >= 0 and (p < 0 or lives[p]))
                sees.append((sees[p] if lives[i] and p >= 0 else frozenset()) | {i})
            mask = torch.zeros(Nt, n, dtype=torch.bool)
            for i in range(Nt):
                if lives[i]:
                    mask[i, :max(0, n - Nt)] = True
                    mask[i, [n - Nt + x for x in sees[i]]] = True
            live, mask = torch.tensor(lives, device=DEV), mask.to(DEV)
            of = torch.arange(n, device=DEV) // c["block"]
            for h in range(c["Hkv"]):
                k = s["kc"][b, h, :n].double() * s["ks"][b, h].double()[of][:, None]
                v = s["vc"][b, h, :n].double() * s["vs"][b, h].double()[of][:, None]
                t = torch.matmul(s["q"][b, h * G:(h + 1) * G].double(), k.T) / math.sqrt(c["d"])
                t = t.masked_fill(~mask, -math.inf)[:, live]
                lse[b, h * G:(h + 1) * G, live] = torch.logsumexp(t, -1)
                o[b, h * G:(h + 1) * G, live] = torch.softmax(t, -1) @ v
        return [o, lse]
    if c["op"] == "evict":
        M, block = c["keep"], c["block"]

        def move(codes, scale):
            nb = _blocks(c, M)
            out = torch.empty(c["B"], c["Hkv"], M, c["d"], dtype=torch.float64, device=DEV)
            now = torch.empty(c["B"], c["Hkv"], nb, dtype=torch.float64, device=DEV)
            for b in range(c["B"]):
                for h in range(c["Hkv"]):
                    rows = s["kept"][b, h].long()
                    of = scale[b, h].double()[rows // block]
                    now[b, h] = torch.nn.functional.pad(of, (0, nb * block - M)).view(nb, block).amax(-1)
                    x = codes[b, h].double()[rows] * of[:, None]
                    to = now[b, h].repeat_interleave(block)[:M, None]
                    out[b, h] = _to_e4m3(x / to)
            return out, now

        return [*move(s["kc"], s["ks"]), *move(s["vc"], s["vs"])]
    return _exact_verify(c, s)


def _exact_verify(c, s):
    """One sequence after another, each node's children in order."""
    import itertools

    parents, tokens, u = s["parents"].tolist(), s["tokens"].tolist(), s["u"].double().tolist()
    accepted, counts, follows = [], [], []
    for b in range(c["B"]):
        path = [0]
        while True:
            n = path[-1]
            p = s["p"][b, n].double()
            q = None if s["q"] is None else s["q"][b, n].double()
            rest, total, hit = p, 1.0, None
            for i in range(n + 1, c["Nt"]):
                if parents[b][i] != n:
                    continue
                x = tokens[b][i]
                qx = 1.0 if q is None else q[x].item()
                if u[b][i] * qx * total < rest[x].item():
                    hit = i
                    break
                if q is None:
                    rest = rest.clone()
                    rest[x] = max(rest[x].item() - total, 0.0)
                else:
                    rest = (rest - total * q).clamp(min=0.0)
                total = math.fsum(rest.tolist())
            if hit is None:
                break
            path.append(hit)
        if not rest.sum().item() > 0.0:  # (nothing is left but by rounding: p itself)
            rest = p
        sums = list(itertools.accumulate(rest.tolist()))
        follows.append(next(x for x, below in enumerate(sums) if below > u[b][0] * sums[-1]))
        accepted.append(path + [-1] * (c["Nt"] - len(path)))
        counts.append(len(path))
    return [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (accepted, counts, follows)]
