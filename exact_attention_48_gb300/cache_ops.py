"""Thin ctypes binding of the operators around the key/value cache: rotary
positions, attention for a tree of drafted tokens, accumulated attention
weight per key, eviction.  As in ``binding.py`` every step runs in the
library's kernels; ``include/fa.h`` defines the calls.

A call runs on the device its tensors are on (all of them the same one), on
that device's current PyTorch stream or on ``stream=``; outputs it allocates
belong to that stream.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from .binding import FA_OK, FaError, library

ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}

# A decode step makes these calls per layer and token, so the checks are kept
# lean: one stride() per tensor, stride arrays built once per layout, and the
# raw stream handle instead of a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream


@functools.lru_cache(maxsize=4096)
def _c_strides(strides):
    """Address of the first three strides as int64, and the array that holds them."""
    a = (ctypes.c_int64 * 3)(*strides[:3])
    return ctypes.addressof(a), a


def _view(name, t, dev=None, shape=None):
    """A [B, H, N, d] bf16 view with contiguous d: its pointer and strides."""
    if not isinstance(t, torch.Tensor) or (t.device != dev if dev is not None else not t.is_cuda):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    st = t.stride()
    if len(st) != 4 or st[3] != 1:
        raise ValueError(f"{name} must be a [B, H, N, d] view with contiguous d")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr(), _c_strides(st)


def _plain(name, t, dtype, shape, dev):
    """A contiguous tensor of the given type, shape and device: its pointer."""
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype is not dtype or t.shape != shape \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {dev}")
    return t.data_ptr()


def _row_ints(name, t, B, N, dev):
    """int32 [B, N] (any batch stride) or [N] (shared by the batch): pointer and batch stride."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.device != dev:
        raise ValueError(f"{name} must be an int32 tensor on {dev}")
    if t.shape not in ((B, N), (N,)) or (N > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({B}, {N}) or ({N},) with contiguous rows")
    return t.data_ptr(), t.stride(0) if t.dim() == 2 and B > 1 else 0


def _lens(t, B, dev):
    return None if t is None else _plain("cache_seqlens", t, torch.int32, (B,), dev)


def _table(inv_freq, dev):
    """Pointer of the frequency table and the columns it turns."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be an fp32 tensor [rot / 2]")
    n = inv_freq.shape[0]
    return _plain("inv_freq", inv_freq, torch.float32, (n,), dev), 2 * n


def _empty(shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(t, need, like):
    """The caller's workspace, or one from PyTorch's allocator (on the launching stream): pointer, bytes, owner."""
    if t is None:
        if not need:
            return None, 0, None
        t = _empty(need, torch.uint8, like.device)
    elif not isinstance(t, torch.Tensor) or t.device != like.device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return t.data_ptr(), t.numel() * t.element_size(), t


def _on(dev, stream, body):
    """body(stream handle) with the tensors' device current and outputs allocated for that stream."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return body(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return body(_raw_stream(dev.index))
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        return body(int(stream.cuda_stream))


def _done(rc, where):
    if rc != FA_OK:
        raise FaError(rc, where)


def _heads(q, k):
    """Shapes of grouped queries q against a cache k."""
    B, H, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if Bk != B or dk != d:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected ({B}, Hkv, Nk, {d})")
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"{H} query heads cannot share {Hkv} cache heads")
    return B, H, Nq, d, Hkv, Nk


def fa_rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                        original_len: int = 4096, fast_turns: float = 32.0, slow_turns: float = 1.0, device=None):
    """(inv_freq fp32 [rot / 2], factor) for fa_rope: the frequencies
    base^(-2i / rot), for longer contexts ``scaling`` "linear" (positions
    divided by ``factor``), "base" (base enlarged) or "by_parts" (only the
    frequencies that turn slowly over ``original_len`` positions divided).
    ``device`` defaults to the current CUDA device."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}, got {scaling!r}")
    table = torch.empty(max(0, int(rot)) // 2, dtype=torch.float32)
    out = ctypes.c_float(0.0)
    _done(library().fa_rope_frequencies(table.data_ptr() or None, ctypes.addressof(out), int(rot), float(base),
                                        ROPE_SCALING[scaling], float(factor), int(original_len), float(fast_turns),
                                        float(slow_turns)), "fa_rope_frequencies")
    return table.to("cuda" if device is None else device), float(out.value)


def _rope(where, names, q, k, inv_freq, positions, interleaved, factor, q_out, k_out, stream):
    qp, qs = _view(names[0], q)
    shape = q.shape
    B, H, N, d = shape
    dev, Hkv, kp, ks = q.device, 0, None, (None, None)
    if k is not None:
        kp, ks = _view(names[1], k, dev)
        Hkv = k.shape[1]
        if k.shape != (B, Hkv, N, d):
            raise ValueError(f"{names[1]} has shape {tuple(k.shape)}, expected ({B}, Hkv, {N}, {d})")
    elif k_out is not None:
        raise ValueError(f"{names[3]} given without {names[1]}")
    freq, rot = _table(inv_freq, dev)
    pos, pos_b = (None, 0) if positions is None else _row_ints("positions", positions, B, N, dev)

    def run(handle):
        qo = _empty(shape, torch.bfloat16, dev) if q_out is None else q_out
        qop, qos = _view(names[2], qo, dev, shape)
        ko, kop, kos = k_out, None, (None, None)
        if k is not None:
            ko = _empty(k.shape, torch.bfloat16, dev) if ko is None else ko
            kop, kos = _view(names[3], ko, dev, k.shape)
        _done(getattr(library(), where)(qp, qs[0], kp, ks[0], qop, qos[0], kop, kos[0], pos, pos_b, freq, B, H, Hkv, N,
                                        d, rot, 1 if interleaved else 0, factor, handle), where)
        return qo, ko

    return _on(dev, stream, run)


def fa_rope(q, k, inv_freq, positions=None, interleaved: bool = False, factor: float = 1.0, q_out=None, k_out=None,
            stream=None):
    """Rotary positions: q [B, H, N, d] and k [B, Hkv, N, d] (or None) views
    with contiguous d, turned in their first 2 * len(inv_freq) columns by
    positions (int32 [B, N] or [N], default 0..N-1) times inv_freq and scaled
    by ``factor``.  ``q_out=q, k_out=k`` rotates in place.  Returns (q_out,
    k_out)."""
    return _rope("fa_rope", ("q", "k", "q_out", "k_out"), q, k, inv_freq, positions, interleaved, factor, q_out,
                 k_out, stream)


def fa_rope_bwd(dq_out, dk_out, inv_freq, positions=None, interleaved: bool = False, factor: float = 1.0, dq=None,
                dk=None, stream=None):
    """Gradients of fa_rope: (dq, dk) of a loss whose gradients with respect
    to fa_rope's outputs are dq_out and dk_out (or None), same arguments
    otherwise."""
    return _rope("fa_rope_bwd", ("dq_out", "dk_out", "dq", "dk"), dq_out, dk_out, inv_freq, positions, interleaved,
                 factor, dq, dk, stream)


def fa_rope_append(q, k, v, k_cache, v_cache, cache_seqlens, inv_freq, positions=None, interleaved: bool = False,
                   factor: float = 1.0, q_out=None, stream=None):
    """The N new tokens of each sequence: q [B, H, N, d] rotated (returned;
    ``q_out=q`` in place), k [B, Hkv, N, d] rotated into k_cache and v copied
    into v_cache [B, Hkv, Nk, d], at the last N of the cache_seqlens[b] rows
    (int32 [B], the new rows counted).  positions default to those rows."""
    qp, qs = _view("q", q)
    shape, dev = q.shape, q.device
    B, H, N, d = shape
    kp, ks = _view("k", k, dev)
    kcp, kcs = _view("k_cache", k_cache, dev)
    Hkv, Nk = k.shape[1], k_cache.shape[2]
    if k.shape != (B, Hkv, N, d) or k_cache.shape != (B, Hkv, Nk, d):
        raise ValueError(f"k and k_cache have shapes {tuple(k.shape)} and {tuple(k_cache.shape)}, expected ({B}, Hkv, "
                         f"{N}, {d}) and ({B}, Hkv, Nk, {d})")
    vp, vs = _view("v", v, dev, k.shape)
    vcp, vcs = _view("v_cache", v_cache, dev, k_cache.shape)
    freq, rot = _table(inv_freq, dev)
    lens = _plain("cache_seqlens", cache_seqlens, torch.int32, (B,), dev)
    pos, pos_b = (None, 0) if positions is None else _row_ints("positions", positions, B, N, dev)

    def run(handle):
        qo = _empty(shape, torch.bfloat16, dev) if q_out is None else q_out
        qop, qos = _view("q_out", qo, dev, shape)
        _done(library().fa_rope_append(qp, qs[0], kp, ks[0], vp, vs[0], qop, qos[0], kcp, kcs[0], vcp, vcs[0], lens,
                                       pos, pos_b, freq, B, H, Hkv, N, Nk, d, rot, 1 if interleaved else 0, factor,
                                       handle), "fa_rope_append")
        return qo

    return _on(dev, stream, run)


def fa_tree_workspace_bytes(B: int, H: int, Hkv: int, Nt: int, Nk: int, d: int) -> int:
    return int(library().fa_tree_workspace_bytes(B, H, Hkv, Nt, Nk, d))


def fa_fwd_tree(q, k, v, parents, cache_seqlens=None, scale: float | None = None, o=None, lse=None, workspace=None,
                stream=None):
    """Attention of a tree of Nt <= 128 drafted tokens per sequence: q
    [B, H, Nt, d] against a cache k, v [B, Hkv, Nk, d] whose last Nt of
    cache_seqlens[b] rows are the tree's nodes.  parents (int32 [B, Nt] or
    [Nt]) holds each node's parent node (before it), -1 for the row before
    the tree, anything else for padding (o = 0, lse = -inf).  A node sees the
    rows before the tree, itself and its ancestors.  Returns (o [B, H, Nt, d]
    bf16, lse [B, H, Nt] fp32)."""
    qp, qs = _view("q", q)
    dev = q.device
    kp, ks = _view("k", k, dev)
    B, H, Nt, d, Hkv, Nk = _heads(q, k)
    vp, vs = _view("v", v, dev, k.shape)
    par, par_b = _row_ints("parents", parents, B, Nt, dev)
    cl = _lens(cache_seqlens, B, dev)

    def run(handle):
        out = _empty(q.shape, torch.bfloat16, dev) if o is None else o
        op, os_ = _view("o", out, dev, q.shape)
        ls = _empty((B, H, Nt), torch.float32, dev) if lse is None else lse
        lp = _plain("lse", ls, torch.float32, (B, H, Nt), dev)
        lib = library()
        ws, ws_bytes, own = _workspace(workspace, lib.fa_tree_workspace_bytes(B, H, Hkv, Nt, Nk, d), q)
        _done(lib.fa_fwd_tree(qp, qs[0], kp, ks[0], vp, vs[0], op, os_[0], lp, par, par_b, cl, B, H, Hkv, Nt, Nk, d,
                              1.0 / math.sqrt(d) if scale is None else scale, ws, ws_bytes, handle), "fa_fwd_tree")
        return out, ls

    return _on(dev, stream, run)


def fa_key_weights_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return int(library().fa_key_weights_workspace_bytes(B, H, Hkv, Nq, Nk, d))


def fa_key_weights(q, k, lse, cache_seqlens=None, causal: bool = False, scale: float | None = None, weights_in=None,
                   weights=None, workspace=None, stream=None):
    """Accumulated attention weight of each cached key: weights [B, Hkv, Nk]
    fp32 = weights_in (or zeros) plus, for the rows j < cache_seqlens[b], the
    sum over the query rows q [B, H, Nq, d] that see j (the last Nq
    positions; causal: up to their own) and the heads that share the cache
    head of exp(scale q.k_j - lse).  ``weights=weights_in`` adds in place.

    lse has to be over the rows that the query sees here: that of fa_fwd and
    fa_fwd_decode with the same ``causal``; of fa_fwd_tree one node's, or a
    chain's with ``causal``.  A tree with branches is weighed once its accepted
    branch has been compacted: that branch's queries and lse, ``causal``."""
    qp, qs = _view("q", q)
    dev = q.device
    kp, ks = _view("k", k, dev)
    B, H, Nq, d, Hkv, Nk = _heads(q, k)
    lp = _plain("lse", lse, torch.float32, (B, H, Nq), dev)
    cl = _lens(cache_seqlens, B, dev)
    shape = (B, Hkv, Nk)
    wi = None if weights_in is None else _plain("weights_in", weights_in, torch.float32, shape, dev)

    def run(handle):
        w = _empty(shape, torch.float32, dev) if weights is None else weights
        wp = _plain("weights", w, torch.float32, shape, dev)
        lib = library()
        ws, ws_bytes, own = _workspace(workspace, lib.fa_key_weights_workspace_bytes(B, H, Hkv, Nq, Nk, d), q)
        _done(lib.fa_key_weights(qp, qs[0], kp, ks[0], lp, wi, wp, cl, B, H, Hkv, Nq, Nk, d, 1 if causal else 0,
                                 1.0 / math.sqrt(d) if scale is None else scale, ws, ws_bytes, handle),
              "fa_key_weights")
        return w

    return _on(dev, stream, run)


def fa_cache_select(weights, keep: int, cache_seqlens=None, first: int = 0, recent: int = 0, kept=None,
                    new_seqlens=None, stream=None):
    """Rows to keep of each cache head, given the weights [B, Hkv, Nk] of
    fa_key_weights: the ``first`` first rows, the ``recent`` last ones and the
    heaviest of the others (ties to the lower row).  Returns (kept int32
    [B, Hkv, keep], ascending, -1 behind a shorter sequence's rows,
    new_seqlens int32 [B])."""
    if not isinstance(weights, torch.Tensor) or not weights.is_cuda or weights.dim() != 3:
        raise TypeError("weights must be an fp32 CUDA tensor [B, Hkv, Nk]")
    B, Hkv, Nk = weights.shape
    dev, keep = weights.device, int(keep)
    wp = _plain("weights", weights, torch.float32, (B, Hkv, Nk), dev)
    cl = _lens(cache_seqlens, B, dev)
    if not 1 <= keep <= Nk:
        raise ValueError(f"keep must be in [1, {Nk}], got {keep}")

    def run(handle):
        rows = _empty((B, Hkv, keep), torch.int32, dev) if kept is None else kept
        lens = _empty((B,), torch.int32, dev) if new_seqlens is None else new_seqlens
        _done(library().fa_cache_select(wp, cl, _plain("kept", rows, torch.int32, (B, Hkv, keep), dev),
                                        _plain("new_seqlens", lens, torch.int32, (B,), dev), B, Hkv, Nk, keep, first,
                                        recent, handle), "fa_cache_select")
        return rows, lens

    return _on(dev, stream, run)


def fa_cache_compact(k, v, kept, weights=None, base=None, k_out=None, v_out=None, weights_out=None, stream=None):
    """Moves rows together: row base[b] + i of k_out, v_out [B, Hkv, Nk_out, d]
    (and weights_out [B, Hkv, Nk_out]) becomes row base[b] + kept[b, h, i] of
    k, v (and weights) where that entry is not negative.  kept: int32
    [B, Hkv, M], or [B, M] for all heads.  Without outputs the cache is
    changed in place (the entries must then ascend, none below its place).
    Rows behind the last place filled keep what they held: set their weights to
    0 before new rows are appended there.  Returns (k_out, v_out,
    weights_out)."""
    kp, ks = _view("k", k)
    B, Hkv, Nk, d = k.shape
    dev = k.device
    vp, vs = _view("v", v, dev, k.shape)
    if k_out is None and v_out is None and weights_out is None:
        k_out, v_out, weights_out = k, v, weights
    if k_out is None or v_out is None or (weights is None) != (weights_out is None):
        raise ValueError("give all outputs (weights_out exactly if weights is given) or none")
    kop, kos = _view("k_out", k_out, dev)
    Nout = k_out.shape[2]
    if k_out.shape != (B, Hkv, Nout, d):
        raise ValueError(f"k_out has shape {tuple(k_out.shape)}, expected ({B}, {Hkv}, Nk_out, {d})")
    vop, vos = _view("v_out", v_out, dev, k_out.shape)
    wi = wo = None
    if weights is not None:
        wi = _plain("weights", weights, torch.float32, (B, Hkv, Nk), dev)
        wo = _plain("weights_out", weights_out, torch.float32, (B, Hkv, Nout), dev)
    if not isinstance(kept, torch.Tensor) or kept.dtype is not torch.int32 or kept.device != dev \
            or kept.dim() not in (2, 3):
        raise ValueError("kept must be an int32 tensor [B, Hkv, M] or [B, M]")
    st, M = kept.stride(), kept.shape[-1]
    if kept.shape not in ((B, Hkv, M), (B, M)) or (M > 1 and st[-1] != 1):
        raise ValueError(f"kept has shape {tuple(kept.shape)}, expected ({B}, {Hkv}, M) or ({B}, M), contiguous lists")
    bp = None if base is None else _plain("base", base, torch.int32, (B,), dev)

    def run(handle):
        _done(library().fa_cache_compact(kp, ks[0], vp, vs[0], wi, kop, kos[0], vop, vos[0], wo, kept.data_ptr(),
                                         st[0], st[1] if len(st) == 3 else 0, bp, B, Hkv, Nk, Nout, M, d, handle),
              "fa_cache_compact")
        return k_out, v_out, weights_out

    return _on(dev, stream, run)
