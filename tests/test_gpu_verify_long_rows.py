"""Verification with one CTA a sequence and vocabularies of more tiles than it has places
for: its tiles are longer than 256 elements then."""
import pytest
import torch

import cache_refs as ref
import fp8_cache_refs as r8
from exact_attention_48_gb300 import fa_tree_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("drafted", [False, True])
def test_many_sequences_of_a_large_vocabulary(drafted):
    g = ref.gen(4200)
    B, Nt, V = 160, 3, 300001           # (a cluster a sequence up to 152; tiles of 512 above 262144)
    p = torch.softmax(torch.randn(B, Nt, V, generator=g, device="cuda"), -1)
    q = torch.softmax(torch.randn(B, Nt, V, generator=g, device="cuda"), -1) if drafted else None
    parents = ref.ints([-1, 0, 0])
    tokens = torch.randint(0, V, (B, Nt), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(B, Nt, generator=g, device="cuda")
    u[:4, 0] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.9999, 0.87], device="cuda")
    acc, num, nxt = fa_tree_verify(parents, tokens, p, q, u)
    for b in (0, 1, 2, 3, 50, 101, 159):
        path, token = r8.verify(parents.tolist(), tokens[b].tolist(), p[b].tolist(), None if q is None else q[b].tolist(),
                                u[b].tolist())
        assert acc[b].tolist() == path + [-1] * (Nt - len(path)) and int(num[b]) == len(path), b
        assert int(nxt[b]) == token, (b, int(nxt[b]), token)
