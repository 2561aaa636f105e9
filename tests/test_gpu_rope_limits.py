"""The rotary calls at the largest batches that the header allows: fewer than
2^24 heads of q, and of k, whatever their sum."""
import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import fa_device_status, fa_rope, fa_rope_append, fa_rope_bwd, fa_rope_frequencies

pytestmark = pytest.mark.gpu


def test_millions_of_sequences():
    B, d = (1 << 23) + 5, 64
    g = ref.gen(700)
    q = torch.empty(B, 1, 1, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    k = torch.empty(B, 1, 1, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    pos = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    freq, _ = fa_rope_frequencies(d)
    some = torch.tensor([0, 1, 77, 1 << 22, (1 << 23) + 1, B - 1], device="cuda")
    want = fa_rope(q[some], k[some], freq, pos[some])
    for call in (fa_rope, fa_rope_bwd):
        got = call(q, k, freq, pos)
        want = call(q[some], k[some], freq, pos[some])
        assert torch.equal(got[0][some], want[0]) and torch.equal(got[1][some], want[1])
    lens = torch.ones(B, device="cuda", dtype=torch.int32)
    kc, vc = torch.zeros_like(k), torch.zeros_like(k)
    qo = fa_rope_append(q, k, q, kc, vc, lens, freq, pos)
    want = fa_rope(q[some], k[some], freq, pos[some])
    assert torch.equal(qo[some], want[0]) and torch.equal(kc[some], want[1]) and torch.equal(vc, q)
    assert fa_device_status() == 0
