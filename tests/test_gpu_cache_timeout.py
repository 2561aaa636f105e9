"""The bounded pipeline waits of the cache operators, on the test build that
test_gpu_timeout.py describes (waits of a millisecond, and each kernel's first
V tile, key block or query tile left out): a call gives up, reports
FA_ERR_DEVICE_TIMEOUT once and leaves the context usable; no role of a block
waits for another that has given up."""
import ctypes
import math

import pytest
import torch

import cache_refs as ref
from exact_attention_48_gb300 import build as fa_build
from exact_attention_48_gb300 import fa_device_status, fa_fwd_tree, fa_key_weights

pytestmark = pytest.mark.gpu

FA_OK, FA_ERR_DEVICE_TIMEOUT = 0, 5


@pytest.fixture(scope="module")
def stall():
    lib = ctypes.CDLL(fa_build.build_variant("stalltest"))
    vp, i, f, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64, ctypes.c_size_t
    lib.fa_fwd_tree.argtypes = [vp] * 10 + [i64, vp] + [i] * 6 + [f, vp, sz, vp]
    lib.fa_key_weights.argtypes = [vp] * 8 + [i] * 7 + [f, vp, sz, vp]
    lib.fa_device_status.argtypes = [vp]
    lib.fa_debug_last_wait_site.argtypes = []
    return lib


def st(t):
    return ctypes.addressof(_keep.setdefault(tuple(t.stride()[:3]), (ctypes.c_int64 * 3)(*t.stride()[:3])))


_keep = {}


def gave_up(lib):
    torch.cuda.synchronize()          # every kernel has returned
    s = torch.cuda.current_stream().cuda_stream
    site = lib.fa_debug_last_wait_site()
    assert lib.fa_device_status(s) == FA_ERR_DEVICE_TIMEOUT and site > 0
    assert lib.fa_device_status(s) == FA_OK     # reported once


# one row tile (two warpgroups that meet at barriers), two of them, many units a run, a cut unit; both d
@pytest.mark.parametrize("B,H,Hkv,Nt,Nk,d", [(1, 2, 2, 5, 300, 128), (2, 8, 2, 64, 3000, 128), (70, 4, 4, 3, 500, 64),
                                             (1, 4, 1, 33, 20000, 64)])
def test_tree(stall, B, H, Hkv, Nt, Nk, d):
    g = ref.gen(300)
    q, k, v = ref.draw(g, B, H, Nt, d), ref.draw(g, B, Hkv, Nk, d), ref.draw(g, B, Hkv, Nk, d)
    par = ref.ints(list(range(-1, Nt - 1)))
    for _ in range(2):
        o, lse = torch.zeros_like(q), torch.zeros(B, H, Nt, device="cuda")
        rc = stall.fa_fwd_tree(q.data_ptr(), st(q), k.data_ptr(), st(k), v.data_ptr(), st(v), o.data_ptr(), st(o),
                               lse.data_ptr(), par.data_ptr(), 0, None, B, H, Hkv, Nt, Nk, d, 1 / math.sqrt(d), None,
                               0, torch.cuda.current_stream().cuda_stream)
        assert rc == FA_OK
        gave_up(stall)
    o, lse = fa_fwd_tree(q, k, v, par)
    assert fa_device_status() == FA_OK and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d", [(2, 2, 2, 1, 3000, 128), (2, 4, 2, 300, 1000, 64),
                                             (4, 16, 16, 200, 2000, 128), (1, 2, 1, 2000, 500, 128)])
def test_key_weights(stall, B, H, Hkv, Nq, Nk, d):
    g = ref.gen(301)
    q, k = ref.draw(g, B, H, Nq, d), ref.draw(g, B, Hkv, Nk, d)
    lse = torch.full((B, H, Nq), 8.0, device="cuda")
    for _ in range(2):
        w = torch.zeros(B, Hkv, Nk, device="cuda")
        rc = stall.fa_key_weights(q.data_ptr(), st(q), k.data_ptr(), st(k), lse.data_ptr(), None, w.data_ptr(), None, B,
                                  H, Hkv, Nq, Nk, d, 1, 0.1, None, 0, torch.cuda.current_stream().cuda_stream)
        assert rc == FA_OK
        gave_up(stall)
    w = fa_key_weights(q, k, lse, None, True, 0.1)
    assert fa_device_status() == FA_OK and bool(torch.isfinite(w).all())
