"""Head counts past the header's limits are refused on the host, before any
CUDA call (the addresses are made up); the largest allowed ones run in
test_gpu_rope_limits.py."""
import ctypes

import pytest

from exact_attention_48_gb300 import build as fa_build
from exact_attention_48_gb300.binding import library

INVALID = 1


def at(n):
    return (1 << 44) + (n << 40)


@pytest.mark.parametrize("B,H,Hkv", [(1 << 20, 16, 1), (1 << 20, 1, 16), (1 << 24, 1, 1), (1, 1 << 24, 1), (1, 1, 1 << 24)])
def test_rope_head_counts(B, H, Hkv):
    fa_build.build()
    lib = library()
    sq, sk = ((ctypes.c_int64 * 3)(h * 64, 64, 64) for h in (H, Hkv))
    for call in (lib.fa_rope, lib.fa_rope_bwd):
        assert call(at(0), sq, at(1), sk, at(2), sq, at(3), sk, None, 0, at(4), B, H, Hkv, 1, 64, 64, 0, 1.0,
                    None) == INVALID
    assert lib.fa_rope_append(at(0), sq, at(1), sk, at(2), sk, at(3), sq, at(4), sk, at(5), sk, at(6), None, 0, at(7), B,
                              H, Hkv, 1, 1, 64, 64, 0, 1.0, None) == INVALID
