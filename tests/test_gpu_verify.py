"""Verification of drafted tokens (fa_tree_verify) against its definition with exact
sums: the same nodes and the same token.  (A number decides otherwise only where it
lies within about 2^-45 of a border, relative to the sums: none of these does.)"""
import math

import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import fa_tree_verify

pytestmark = pytest.mark.gpu


def dist(g, B, Nt, V, sharp):
    return torch.softmax(sharp * torch.randn(B, Nt, V, generator=g, device="cuda"), -1)


def tree_of(g, B, Nt, wide):
    i = torch.arange(Nt, device="cuda")
    u = torch.rand(B, Nt, generator=g, device="cuda") ** (3.0 if wide else 0.5)
    parents = torch.minimum((u * i).floor(), (i - 1).float()).to(torch.int32)
    parents[:, 0] = -1
    return parents


def check(parents, tokens, p, q, u, got=None):
    acc, num, nxt = fa_tree_verify(parents, tokens, p, q, u) if got is None else got
    B, Nt, V = p.shape
    row = lambda t, b: t[b].tolist() if t.dim() == 2 else t.tolist()  # noqa: E731
    for b in range(B):
        path, token = r8.verify(row(parents, b), row(tokens, b), p[b].tolist(), None if q is None else q[b].tolist(),
                                row(u, b))
        assert acc[b].tolist() == path + [-1] * (Nt - len(path)), f"b{b}"
        assert int(num[b]) == len(path) and int(nxt[b]) == token, f"b{b}: {int(nxt[b])} {token}"


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("B,Nt,V,wide", [
    (1, 1, 1, False), (3, 1, 7, False), (8, 5, 2, True), (16, 8, 33, False), (16, 12, 257, True), (4, 6, 4096, False),
    (4, 10, 4097, True), (3, 16, 10001, True), (2, 128, 300, True), (40, 4, 600, True),
])
def test_random_trees(B, Nt, V, wide, drafted):
    g = ref.gen(4000 + V + Nt)
    p = dist(g, B, Nt, V, 2.0)
    q = dist(g, B, Nt, V, 2.0) if drafted else None
    if drafted:
        q[::2] = p[::2] * 0.7 + q[::2] * 0.3
    parents = tree_of(g, B, Nt, wide)
    u = torch.rand(B, Nt, generator=g, device="cuda")
    # half of the tokens likely ones, so that some are accepted
    likely = p.gather(1, parents.clamp(min=0).long()[..., None].expand(-1, -1, V)).argmax(-1)
    tokens = torch.where(torch.rand(B, Nt, generator=g, device="cuda") < 0.5, likely,
                         torch.randint(0, V, (B, Nt), generator=g, device="cuda")).to(torch.int32)
    check(parents, tokens, p, q, u)


def test_large_vocabulary():
    g = ref.gen(4001)
    p, q = dist(g, 2, 4, 131072, 3.0), dist(g, 2, 4, 131072, 3.0)
    parents = ref.ints([[-1, 0, 0, 0], [-1, 0, 1, 2]])
    tokens = torch.randint(0, 131072, (2, 4), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(2, 4, generator=g, device="cuda")
    check(parents, tokens, p, q, u)
    check(parents, tokens, p, None, u)
    p = dist(g, 1, 2, 1000003, 1.0)
    check(ref.ints([-1, 0]), ref.ints([0, 77]), p, p * 0.9, torch.rand(2, generator=g, device="cuda"))


def test_numbers_at_their_ends():
    g = ref.gen(4002)
    p, q = dist(g, 4, 3, 50, 1.0), dist(g, 4, 3, 50, 1.0)
    p[1, :, :20] = 0.0     # the first tokens have no mass
    p[1, :, 45:] = 0.0
    p[2] = q[2]            # the same distribution: always accepted
    parents = tree_of(g, 4, 3, True)
    tokens = torch.randint(0, 50, (4, 3), generator=g, device="cuda", dtype=torch.int32)
    for value in (0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24):
        u = torch.full((4, 3), value, device="cuda")
        check(parents, tokens, p, q, u)
        check(parents, tokens, p, None, u)
    acc, num, nxt = fa_tree_verify(ref.ints([-1, 0, 1]), tokens, p, q, torch.full((3,), 1 - 2.0 ** -24, device="cuda"))
    assert int(num[2]) == 3


def test_certain_rows():
    """One-hot target rows (greedy): the child with that token is accepted whatever its number; else the token follows.
    The same with the draft's rows like them: a child of no probability takes all that is left, and the target's row
    takes its place."""
    p = torch.zeros(2, 4, 9, device="cuda")
    p[:, 0, 3] = p[:, 1, 5] = p[:, 2, 1] = p[:, 3, 8] = 1.0
    parents, u = ref.ints([-1, 0, 0, 2]), torch.tensor([0.999, 0.999, 0.999, 0.0], device="cuda")
    tokens = ref.ints([[0, 2, 3, 1], [0, 2, 3, 4]])
    acc, num, nxt = fa_tree_verify(parents, tokens, p, None, u)
    assert acc.tolist() == [[0, 2, 3, -1], [0, 2, -1, -1]] and num.tolist() == [3, 2] and nxt.tolist() == [8, 1]
    acc, num, nxt = fa_tree_verify(parents, tokens, p, p, u)
    assert acc.tolist() == [[0, -1, -1, -1]] * 2 and num.tolist() == [1, 1] and nxt.tolist() == [3, 3]
    check(parents, tokens, p, p, u)


def test_padding_and_invalid_nodes():
    g = ref.gen(4003)
    p, q = dist(g, 6, 6, 100, 2.0), dist(g, 6, 6, 100, 2.0)
    parents = ref.ints([[-1, 0, -2, 1, 5, 3], [-2, 0, 0, 0, 0, 0], [-1, -1, -1, 0, 0, 4], [0, 0, 1, 1, 1, 1],
                        [-1, 0, 1, 1, 9, 0], [-1, 1, 0, 3, 2, 2]])
    tokens = torch.randint(0, 100, (6, 6), generator=g, device="cuda", dtype=torch.int32)
    tokens[0, 1], tokens[4, 1], tokens[5, 2] = 100, -1, -(1 << 31)
    u = 0.3 * torch.rand(6, 6, generator=g, device="cuda")
    check(parents, tokens, p, q, u)
    check(parents, tokens, p, None, u)


def test_nothing_to_draw_from():
    p = torch.zeros(2, 2, 5000, device="cuda")
    p[1, 0, 17] = 0.25       # not normalised: its sum counts
    acc, num, nxt = fa_tree_verify(ref.ints([-1, 0]), ref.ints([0, 3]), p, None, torch.tensor([0.9, 0.5], device="cuda"))
    assert nxt.tolist() == [-1, 17] and num.tolist() == [1, 1]


def test_strides_shared_rows_and_outputs():
    g = ref.gen(4004)
    big = dist(g, 3, 5, 210, 2.0)
    p, q = big[:, :, 3:104], big[:, :, 105:206]
    parents = tree_of(g, 3, 9, True)[:, 2:7]
    parents = torch.where(parents >= 5, torch.zeros_like(parents), parents)
    parents = torch.cat([torch.full((3, 1), -1, device="cuda", dtype=torch.int32), parents[:, 1:].clamp(max=0)], 1)
    tokens = torch.randint(0, 101, (3, 8), generator=g, device="cuda", dtype=torch.int32)[:, 1:6]
    u = torch.rand(3, 11, generator=g, device="cuda")[:, 3:8]
    check(parents, tokens, p, q, u)
    check(parents, tokens, p, big[:1, :1, 105:206].expand(3, 5, 101), u)
    shared = ref.ints([-1, 0, 0, 1, 1])
    check(shared, tokens[0], p, q, u[1])
    out = [torch.full((3, 5), 9, dtype=torch.int32, device="cuda")] + [torch.full((3,), 9, dtype=torch.int32, device="cuda") for _ in range(2)]
    got = fa_tree_verify(shared, tokens, p, q, u, *out)
    assert all(a is b for a, b in zip(got, out))
    check(shared, tokens, p, q, u, got)


def test_tokens_follow_the_target():
    """The first token behind the root (accepted or the next one) is distributed as the target's, whatever was drafted:
    frequencies of 40000 sequences within five standard deviations."""
    g = ref.gen(4005)
    B, V = 40000, 6
    p1, q1 = torch.softmax(torch.randn(2, V, generator=g, device="cuda"), -1)
    p, q = p1.expand(B, 4, V).contiguous(), q1.expand(B, 4, V).contiguous()
    tokens = torch.multinomial(q1.expand(B, V), 4, replacement=True, generator=g).to(torch.int32)
    parents = ref.ints([-1, 0, 0, 0])
    u = torch.rand(B, 4, generator=g, device="cuda")
    acc, num, nxt = fa_tree_verify(parents, tokens, p, q, u)
    first = torch.where(num > 1, tokens.gather(1, acc[:, 1:2].clamp(min=0).long())[:, 0], nxt)
    freq = torch.bincount(first.long(), minlength=V).double() / B
    sd = (p1.double() * (1 - p1.double()) / B).sqrt()
    assert bool(((freq - p1.double()).abs() <= 5 * sd).all()), (freq, p1)
    # without the draft's probabilities: the same tokens for all
    acc, num, nxt = fa_tree_verify(parents, ref.ints([0, 2, 2, 4]), p, None, u)
    first = torch.where(num > 1, ref.ints([0, 2, 2, 4])[acc[:, 1].clamp(min=0).long()], nxt)
    freq = torch.bincount(first.long(), minlength=V).double() / B
    assert bool(((freq - p1.double()).abs() <= 5 * sd).all()), (freq, p1)


def test_graph_streams_and_refusals():
    g = ref.gen(4006)
    p, q = dist(g, 5, 6, 20000, 2.0), dist(g, 5, 6, 20000, 2.0)
    parents = tree_of(g, 5, 6, True)
    tokens = torch.randint(0, 20000, (5, 6), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(5, 6, generator=g, device="cuda")
    want = fa_tree_verify(parents, tokens, p, q, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa_tree_verify(parents, tokens, p, q, u, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa_tree_verify(parents, tokens, p, q, u)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, out):
        assert torch.equal(a, b) and torch.equal(a, c)
    for bad in (dict(parents=parents.long()), dict(tokens=tokens[:, :5]), dict(target=p.double()), dict(target=p.cpu()),
                dict(draft=q[:, :, :100]), dict(draft=q.half()), dict(uniforms=u.double()), dict(uniforms=u[:2])):
        a = {**dict(parents=parents, tokens=tokens, target=p, draft=q, uniforms=u), **bad}
        with pytest.raises((TypeError, ValueError)):
            fa_tree_verify(**a)
