"""Key weights of many query rows where a block works through several units:
every key against 64 bits, within the bound of test_gpu_key_weights.py.  The
shapes have more 256-key units than twice the GPU's multiprocessors (units of
that many are not split), so that the rings of keys, queries and scores, the
sums' buffer and the order of the units go on from unit to unit."""
import math

import pytest
import torch

import cache_refs as ref
import test_gpu_key_weights as kw
from exact_attention_48_gb300 import fa_device_status, fa_key_weights, fa_key_weights_workspace_bytes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,layout", [
    (4, 16, 16, 200, 2000, 128, "bhnd"),    # 512 units of two query tiles
    (4, 16, 16, 200, 2000, 64, "bnhd"),
    (8, 16, 8, 100, 1500, 128, "bnhd"),     # two heads of a tile each, 384 units
    (5, 24, 8, 30, 2100, 64, "bhnd"),       # heads packed into a tile, 360 units
    (3, 30, 10, 300, 3100, 64, "pitch"),    # three heads of three tiles, 390 units
    (1, 64, 64, 4096, 1025, 128, "bhnd"),   # heads in windows of 48: 48 and 16
    (2, 64, 64, 4096, 1025, 64, "bhnd"),    # 128 heads in windows of 96: 96 and 32
])
def test_units_in_turn(B, H, Hkv, Nq, Nk, d, layout, causal):
    g = ref.gen(500 + Nk + Nq)
    assert B * Hkv * ((Nk + 255) // 256) >= 304 and fa_key_weights_workspace_bytes(B, H, Hkv, Nq, Nk, d) == 0
    scale = 1 / math.sqrt(d)
    q, k = ref.draw(g, B, H, Nq, d, layout), ref.draw(g, B, Hkv, Nk, d, layout)
    # (the causal lengths below Nq leave units, and whole sequences, that few rows or none see)
    lens = ([Nk, Nk - Nk // 3, Nq, Nk // 3, 0] * B)[:B]
    lse = kw.lse_of(q, k, lens, causal, scale)
    w_in = torch.rand(B, Hkv, Nk, generator=g, device="cuda")
    w = fa_key_weights(q, k, lse, ref.ints(lens), causal, weights_in=w_in)
    assert fa_device_status() == 0
    kw.check(q, k, lse, w_in, w, lens, causal, scale, f"Nq{Nq} Nk{Nk}")


@pytest.mark.parametrize("Nq,d", [(1, 128), (33, 64), (700, 128), (700, 64)])
def test_first_results_of_the_repeated_launches(Nq, d):
    """The shapes, draws and lengths that test_weights_and_eviction_under_load repeats."""
    g = ref.gen(99)
    B, H, Hkv, Nk = 3, 8, 4, 5000
    q, k = ref.draw(g, B, H, Nq, d), ref.draw(g, B, Hkv, Nk, d)
    lens = [5000, 4097, 900]
    lse = torch.rand(B, H, Nq, generator=g, device="cuda") + 8
    w = fa_key_weights(q, k, lse, ref.ints(lens), True)
    assert fa_device_status() == 0
    kw.check(q, k, lse, None, w, lens, True, 1 / math.sqrt(d), f"Nq{Nq}")
