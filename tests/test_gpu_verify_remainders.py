"""Verification without the draft's probabilities where rejected children take almost
all that is left: what remains decides as in the definition."""
import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import fa_tree_verify
from test_gpu_verify import check

pytestmark = pytest.mark.gpu

LAST = 1 - 2.0 ** -24       # the greatest number below 1 that fp32 uniforms take


@pytest.mark.parametrize("V", [6, 5000, 40000])
def test_children_that_leave_next_to_nothing(V):
    """p = a, b, b r, b r^2, b r^3 with r = 1.5 * 2^-24, and nothing else: with the number LAST each child before the last
    is rejected (LAST * (1 + r) > 1), and the last one, which has all that is left, accepted, as
    LAST * S < S. S falls by a factor of 2^-23.4 a child, below the last place of the first sum's 48 bits."""
    g = ref.gen(4100 + V)
    B = 300 if V < 40000 else 24
    p = torch.zeros(B, 6, V, device="cuda")
    at = torch.rand(B, V, generator=g, device="cuda").argsort(-1)[:, :5]
    a = 0.25 + 0.25 * torch.rand(B, generator=g, device="cuda")
    b = (1.0 - a) * (0.5 + 0.5 * torch.rand(B, generator=g, device="cuda"))
    seq = torch.arange(B, device="cuda")
    r = 1.5 * 2.0 ** -24
    for i, x in enumerate((a, b, b * r, b * r * r, b * r * r * r)):
        p[seq, 0, at[:, i]] = x * (1.0 if i == 0 else (1.0 + 0.01 * torch.rand(B, generator=g, device="cuda")))
    p[:, 1:, 0] = 1.0
    parents = ref.ints([-1, 0, 0, 0, 0, 0])
    tokens = torch.cat([torch.zeros(B, 1, device="cuda", dtype=torch.int64), at], 1).to(torch.int32)
    u = torch.tensor([0.5] + [LAST] * 5, device="cuda")
    got = fa_tree_verify(parents, tokens, p, None, u)
    assert bool((got[1] == 2).all()) and bool((got[0][:, 1] == 5).all())
    check(parents, tokens, p, None, u, got)


def test_a_token_of_no_probability_is_never_accepted():
    """Six children: the last has no probability, and the one before it almost none, whatever is left of the sums."""
    g = ref.gen(4110)
    B, V, Nt = 2000, 12, 7
    p = torch.rand(B, Nt, V, generator=g, device="cuda") * torch.exp2(torch.randint(-30, 1, (B, Nt, V), generator=g,
                                                                                      device="cuda").float())
    order = p[:, 0].argsort(-1, descending=True)
    p = p / p.sum(-1, keepdim=True)
    tokens = torch.cat([order[:, :1], order[:, :6]], 1)
    p[torch.arange(B, device="cuda"), 0, tokens[:, 6]] = 0.0
    parents, u = ref.ints([-1, 0, 0, 0, 0, 0, 0]), torch.full((Nt,), LAST, device="cuda")
    got = fa_tree_verify(parents, tokens.to(torch.int32), p, None, u)
    assert not bool((got[0][:, 1] == 6).any())
    check(parents, tokens.to(torch.int32), p, None, u, got)


def test_the_same_token_twice():
    """A child whose token was rejected before has nothing left: it is rejected whatever its number."""
    g = ref.gen(4120)
    B, V = 500, 300
    p = torch.softmax(3.0 * torch.randn(B, 6, V, generator=g, device="cuda"), -1)
    best = p[:, 0].topk(2)[1]
    tokens = best[:, [0, 0, 0, 1, 0, 1]].to(torch.int32)
    parents = ref.ints([-1, 0, 0, 0, 0, 0])
    for value in (0.0, 0.5, 0.97, LAST):
        u = torch.rand(B, 6, generator=g, device="cuda")
        u[:, 2] = u[:, 4] = value
        check(parents, tokens, p, None, u)
