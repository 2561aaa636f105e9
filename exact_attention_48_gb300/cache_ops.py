"""Thin ctypes binding of the operators around the key/value cache: rotary
positions, attention for a tree of drafted tokens, accumulated attention
weight per key, eviction.  As in ``binding.py`` every step runs in the
library's kernels; ``include/fa.h`` defines the calls.

A call runs on the device its tensors are on (all of them the same one), on
that device's current PyTorch stream or on ``stream=``; outputs it allocates
belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import torch

from .binding import FA_OK, FaError, _check_view, library

ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}


@functools.lru_cache(maxsize=4096)
def _c_strides(strides):
    return (ctypes.c_int64 * 3)(*strides)


def _strides(t):
    return _c_strides(t.stride()[:3])


def _check_plain(name, t, dtype, shape, device):
    """A contiguous tensor of the given type, shape and device."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != dtype or tuple(t.shape) != tuple(shape) \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {device}")
    return t


def _check_views(device, **views):
    for name, (t, shape) in views.items():
        _check_view(name, t, shape)
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _row_ints(name, t, B, N, device):
    """int32 [B, N] (any batch stride) or [N] (shared by the batch): pointer and batch stride."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise ValueError(f"{name} must be an int32 tensor on {device}")
    if tuple(t.shape) not in ((B, N), (N,)) or (N > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({B}, {N}) or ({N},) with contiguous rows")
    return t.data_ptr(), t.stride(0) if t.dim() == 2 and B > 1 else 0


def _lens(t, B, device):
    return None if t is None else _check_plain("cache_seqlens", t, torch.int32, (B,), device).data_ptr()


def _workspace(t, device):
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return t.data_ptr(), t.numel() * t.element_size()


@contextlib.contextmanager
def _on(device, stream):
    """The tensors' device made current, and the stream (its handle) that outputs are allocated for."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with contextlib.ExitStack() as stack:
        if torch.cuda.current_device() != device.index:
            stack.enter_context(torch.cuda.device(device))
        if stream is not None:
            stack.enter_context(torch.cuda.stream(stream))
        else:
            stream = torch.cuda.current_stream(device)
        yield int(stream.cuda_stream)


def _done(rc, where):
    if rc != FA_OK:
        raise FaError(rc, where)


def _heads(q, k, names=("q", "k")):
    """Shapes of grouped queries against a cache: B, H, Nq, d, Hkv, Nk."""
    _check_view(names[0], q)
    _check_view(names[1], k)
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"{names[1]} has shape {tuple(k.shape)}, expected ({B}, Hkv, Nk, {d})")
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
    _check_view(names[0], q)
    B, H, N, d = q.shape
    dev, Hkv = q.device, 0
    if k is not None:
        _check_view(names[1], k)
        Hkv = k.shape[1]
        _check_views(dev, **{names[1]: (k, (B, Hkv, N, d))})
    elif k_out is not None:
        raise ValueError(f"{names[3]} given without {names[1]}")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be an fp32 tensor [rot / 2]")
    rot = 2 * inv_freq.shape[0]
    _check_plain("inv_freq", inv_freq, torch.float32, (rot // 2,), dev)
    pos, pos_b = (None, 0) if positions is None else _row_ints("positions", positions, B, N, dev)
    with _on(dev, stream) as handle:
        q_out = torch.empty(q.shape, device=dev, dtype=q.dtype) if q_out is None else q_out
        _check_views(dev, **{names[2]: (q_out, q.shape)})
        kp = kop = ks = kos = None
        if k is not None:
            k_out = torch.empty(k.shape, device=dev, dtype=k.dtype) if k_out is None else k_out
            _check_views(dev, **{names[3]: (k_out, k.shape)})
            kp, ks, kop, kos = k.data_ptr(), _strides(k), k_out.data_ptr(), _strides(k_out)
        _done(getattr(library(), where)(q.data_ptr(), _strides(q), kp, ks, q_out.data_ptr(), _strides(q_out), kop, kos,
                                        pos, pos_b, inv_freq.data_ptr(), B, H, Hkv, N, d, rot, int(bool(interleaved)),
                                        float(factor), handle), where)
    return q_out, k_out


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
    _check_view("q", q)
    B, H, N, d = q.shape
    dev = q.device
    _check_view("k", k)
    _check_view("k_cache", k_cache)
    Hkv, Nk = k.shape[1], k_cache.shape[2]
    _check_views(dev, k=(k, (B, Hkv, N, d)), v=(v, (B, Hkv, N, d)), k_cache=(k_cache, (B, Hkv, Nk, d)),
                 v_cache=(v_cache, (B, Hkv, Nk, d)))
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be an fp32 tensor [rot / 2]")
    rot = 2 * inv_freq.shape[0]
    _check_plain("inv_freq", inv_freq, torch.float32, (rot // 2,), dev)
    _check_plain("cache_seqlens", cache_seqlens, torch.int32, (B,), dev)
    pos, pos_b = (None, 0) if positions is None else _row_ints("positions", positions, B, N, dev)
    with _on(dev, stream) as handle:
        q_out = torch.empty(q.shape, device=dev, dtype=q.dtype) if q_out is None else q_out
        _check_views(dev, q_out=(q_out, q.shape))
        _done(library().fa_rope_append(
            q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), v.data_ptr(), _strides(v), q_out.data_ptr(),
            _strides(q_out), k_cache.data_ptr(), _strides(k_cache), v_cache.data_ptr(), _strides(v_cache),
            cache_seqlens.data_ptr(), pos, pos_b, inv_freq.data_ptr(), B, H, Hkv, N, Nk, d, rot,
            int(bool(interleaved)), float(factor), handle), "fa_rope_append")
    return q_out


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
    B, H, Nt, d, Hkv, Nk = _heads(q, k)
    dev = q.device
    _check_views(dev, k=(k, k.shape), v=(v, k.shape))
    par, par_b = _row_ints("parents", parents, B, Nt, dev)
    cl = _lens(cache_seqlens, B, dev)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    ws, ws_bytes = _workspace(workspace, dev)
    with _on(dev, stream) as handle:
        o = torch.empty(q.shape, device=dev, dtype=q.dtype) if o is None else o
        _check_views(dev, o=(o, q.shape))
        lse = torch.empty((B, H, Nt), device=dev, dtype=torch.float32) if lse is None else lse
        _check_plain("lse", lse, torch.float32, (B, H, Nt), dev)
        _done(library().fa_fwd_tree(q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), v.data_ptr(), _strides(v),
                                    o.data_ptr(), _strides(o), lse.data_ptr(), par, par_b, cl, B, H, Hkv, Nt, Nk, d,
                                    float(scale), ws, ws_bytes, handle), "fa_fwd_tree")
    return o, lse


def fa_key_weights_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return int(library().fa_key_weights_workspace_bytes(B, H, Hkv, Nq, Nk, d))


def fa_key_weights(q, k, lse, cache_seqlens=None, causal: bool = False, scale: float | None = None, weights_in=None,
                   weights=None, workspace=None, stream=None):
    """Accumulated attention weight of each cached key: weights [B, Hkv, Nk]
    fp32 = weights_in (or zeros) plus, for the rows j < cache_seqlens[b], the
    sum over the query rows q [B, H, Nq, d] that see j (the last Nq
    positions; causal: up to their own) and the heads that share the cache
    head of exp(scale q.k_j - lse).  ``weights=weights_in`` adds in place."""
    B, H, Nq, d, Hkv, Nk = _heads(q, k)
    dev = q.device
    _check_views(dev, k=(k, k.shape))
    _check_plain("lse", lse, torch.float32, (B, H, Nq), dev)
    cl = _lens(cache_seqlens, B, dev)
    if weights_in is not None:
        _check_plain("weights_in", weights_in, torch.float32, (B, Hkv, Nk), dev)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    ws, ws_bytes = _workspace(workspace, dev)
    with _on(dev, stream) as handle:
        weights = torch.empty((B, Hkv, Nk), device=dev, dtype=torch.float32) if weights is None else weights
        _check_plain("weights", weights, torch.float32, (B, Hkv, Nk), dev)
        _done(library().fa_key_weights(q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), lse.data_ptr(),
                                       None if weights_in is None else weights_in.data_ptr(), weights.data_ptr(), cl,
                                       B, H, Hkv, Nq, Nk, d, int(bool(causal)), float(scale), ws, ws_bytes, handle),
              "fa_key_weights")
    return weights


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
    _check_plain("weights", weights, torch.float32, (B, Hkv, Nk), dev)
    cl = _lens(cache_seqlens, B, dev)
    if not 1 <= keep <= Nk:
        raise ValueError(f"keep must be in [1, {Nk}], got {keep}")
    with _on(dev, stream) as handle:
        kept = torch.empty((B, Hkv, keep), device=dev, dtype=torch.int32) if kept is None else kept
        _check_plain("kept", kept, torch.int32, (B, Hkv, keep), dev)
        new_seqlens = torch.empty(B, device=dev, dtype=torch.int32) if new_seqlens is None else new_seqlens
        _check_plain("new_seqlens", new_seqlens, torch.int32, (B,), dev)
        _done(library().fa_cache_select(weights.data_ptr(), cl, kept.data_ptr(), new_seqlens.data_ptr(), B, Hkv, Nk,
                                        keep, int(first), int(recent), handle), "fa_cache_select")
    return kept, new_seqlens


def fa_cache_compact(k, v, kept, weights=None, base=None, k_out=None, v_out=None, weights_out=None, stream=None):
    """Moves rows together: row base[b] + i of k_out, v_out [B, Hkv, Nk_out, d]
    (and weights_out [B, Hkv, Nk_out]) becomes row base[b] + kept[b, h, i] of
    k, v (and weights) where that entry is not negative.  kept: int32
    [B, Hkv, M], or [B, M] for all heads.  Without outputs the cache is
    changed in place (the entries must then ascend, none below its place).
    Returns (k_out, v_out, weights_out)."""
    _check_view("k", k)
    B, Hkv, Nk, d = k.shape
    dev = k.device
    _check_views(dev, v=(v, k.shape))
    if k_out is None and v_out is None and weights_out is None:
        k_out, v_out, weights_out = k, v, weights
    if k_out is None or v_out is None or (weights is None) != (weights_out is None):
        raise ValueError("give all outputs (weights_out exactly if weights is given) or none")
    _check_view("k_out", k_out)
    Nout = k_out.shape[2]
    _check_views(dev, k_out=(k_out, (B, Hkv, Nout, d)), v_out=(v_out, (B, Hkv, Nout, d)))
    wi = wo = None
    if weights is not None:
        wi = _check_plain("weights", weights, torch.float32, (B, Hkv, Nk), dev).data_ptr()
        wo = _check_plain("weights_out", weights_out, torch.float32, (B, Hkv, Nout), dev).data_ptr()
    if not isinstance(kept, torch.Tensor) or kept.dtype != torch.int32 or kept.device != dev or kept.dim() not in (2, 3):
        raise ValueError("kept must be an int32 tensor [B, Hkv, M] or [B, M]")
    M = kept.shape[-1]
    if tuple(kept.shape) not in ((B, Hkv, M), (B, M)) or (M > 1 and kept.stride(-1) != 1):
        raise ValueError(f"kept has shape {tuple(kept.shape)}, expected ({B}, {Hkv}, M) or ({B}, M), contiguous lists")
    kb, kh = kept.stride(0), kept.stride(1) if kept.dim() == 3 else 0
    bp = None if base is None else _check_plain("base", base, torch.int32, (B,), dev).data_ptr()
    with _on(dev, stream) as handle:
        _done(library().fa_cache_compact(k.data_ptr(), _strides(k), v.data_ptr(), _strides(v), wi, k_out.data_ptr(),
                                         _strides(k_out), v_out.data_ptr(), _strides(v_out), wo, kept.data_ptr(), kb,
                                         kh, bp, B, Hkv, Nk, Nout, M, d, handle), "fa_cache_compact")
    return k_out, v_out, weights_out
