"""Thin ctypes binding of the operators on a cache held in 8 bits (the append of
new rows, attention, rows moved together) and of the verification of drafted
tokens.  As in ``binding.py`` every step runs in the library's kernels;
``include/fa.h`` defines the calls, and streams, devices and outputs are as in
``cache_ops.py``.

A cache in 8 bits is k and v as float8_e4m3fn [B, Hkv, Nk, d] and k_scale and
v_scale, fp32 [B, Hkv, ceil(Nk / block)]: row n of a head stands for its codes
times the scale of block n // block (16, 32, 64 or 128 rows), a power of two.
"""
from __future__ import annotations

import math

import torch

from .binding import library
from .cache_ops import _c_strides, _done, _empty, _heads, _lens, _on, _plain, _row_ints, _table, _view, _workspace


def _view8(name, t, dev, shape=None):
    """A [B, H, N, d] e4m3 view with contiguous d: its pointer and strides."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"{name} must be float8_e4m3fn, got {t.dtype}")
    st = t.stride()
    if len(st) != 4 or st[3] != 1:
        raise ValueError(f"{name} must be a [B, H, N, d] view with contiguous d")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr(), _c_strides(st)


def _scale(name, t, B, Hkv, Nk, block, dev):
    return _plain(name, t, torch.float32, (B, Hkv, -(-Nk // block)), dev)


def _block(block):
    if block not in (16, 32, 64, 128):
        raise ValueError(f"block must be 16, 32, 64 or 128, got {block!r}")
    return int(block)


def fa_rope_append_fp8(q, k, v, k_cache, v_cache, k_scale, v_scale, cache_seqlens, inv_freq, positions=None,
                       interleaved: bool = False, factor: float = 1.0, block: int = 64, q_out=None, stream=None):
    """fa_rope_append to a cache held in 8 bits: the N new tokens of each
    sequence, q [B, H, N, d] rotated (returned; ``q_out=q`` in place), k
    [B, Hkv, N, d] rotated and v rounded into k_cache and v_cache, at the last N
    of the cache_seqlens[b] rows (int32 [B], the new rows counted).  A block
    that gets rows takes the least scale that they fit, or keeps its own if
    that is greater and rows before them use it; where it grows, those rows'
    codes are rounded to it."""
    qp, qs = _view("q", q)
    shape, dev = q.shape, q.device
    B, H, N, d = shape
    block = _block(block)
    kp, ks = _view("k", k, dev)
    kcp, kcs = _view8("k_cache", k_cache, dev)
    Hkv, Nk = k.shape[1], k_cache.shape[2]
    if k.shape != (B, Hkv, N, d) or k_cache.shape != (B, Hkv, Nk, d):
        raise ValueError(f"k and k_cache have shapes {tuple(k.shape)} and {tuple(k_cache.shape)}, expected ({B}, Hkv, "
                         f"{N}, {d}) and ({B}, Hkv, Nk, {d})")
    vp, vs = _view("v", v, dev, k.shape)
    vcp, vcs = _view8("v_cache", v_cache, dev, k_cache.shape)
    ksp = _scale("k_scale", k_scale, B, Hkv, Nk, block, dev)
    vsp = _scale("v_scale", v_scale, B, Hkv, Nk, block, dev)
    freq, rot = _table(inv_freq, dev)
    lens = _plain("cache_seqlens", cache_seqlens, torch.int32, (B,), dev)
    pos, pos_b = (None, 0) if positions is None else _row_ints("positions", positions, B, N, dev)

    def run(handle):
        qo = _empty(shape, torch.bfloat16, dev) if q_out is None else q_out
        qop, qos = _view("q_out", qo, dev, shape)
        _done(library().fa_rope_append_fp8(qp, qs[0], kp, ks[0], vp, vs[0], qop, qos[0], kcp, kcs[0], vcp, vcs[0], ksp,
                                           vsp, lens, pos, pos_b, freq, B, H, Hkv, N, Nk, d, rot,
                                           1 if interleaved else 0, factor, block, handle), "fa_rope_append_fp8")
        return qo

    return _on(dev, stream, run)


def fa_tree_fp8_workspace_bytes(B: int, H: int, Hkv: int, Nt: int, Nk: int, d: int) -> int:
    return int(library().fa_tree_fp8_workspace_bytes(B, H, Hkv, Nt, Nk, d))


def fa_fwd_tree_fp8(q, k, v, k_scale, v_scale, parents=None, cache_seqlens=None, scale: float | None = None,
                    block: int = 64, o=None, lse=None, workspace=None, stream=None):
    """Attention of the last Nt <= 128 rows of each sequence over a cache held
    in 8 bits: q [B, H, Nt, d] bf16 against k, v.  Without ``parents`` each row
    sees the rows up to its own (Nt = 1: a decode step); with them (as for
    fa_fwd_tree) the rows are a tree of drafted tokens.  Returns (o [B, H, Nt, d]
    bf16, lse [B, H, Nt] fp32)."""
    qp, qs = _view("q", q)
    dev = q.device
    kp, ks = _view8("k", k, dev)
    B, H, Nt, d, Hkv, Nk = _heads(q, k)
    vp, vs = _view8("v", v, dev, k.shape)
    block = _block(block)
    ksp = _scale("k_scale", k_scale, B, Hkv, Nk, block, dev)
    vsp = _scale("v_scale", v_scale, B, Hkv, Nk, block, dev)
    par, par_b = (None, 0) if parents is None else _row_ints("parents", parents, B, Nt, dev)
    cl = _lens(cache_seqlens, B, dev)

    def run(handle):
        out = _empty(q.shape, torch.bfloat16, dev) if o is None else o
        op, os_ = _view("o", out, dev, q.shape)
        ls = _empty((B, H, Nt), torch.float32, dev) if lse is None else lse
        lp = _plain("lse", ls, torch.float32, (B, H, Nt), dev)
        lib = library()
        ws, ws_bytes, own = _workspace(workspace, lib.fa_tree_fp8_workspace_bytes(B, H, Hkv, Nt, Nk, d), q)
        _done(lib.fa_fwd_tree_fp8(qp, qs[0], kp, ks[0], vp, vs[0], ksp, vsp, op, os_[0], lp, par, par_b, cl, B, H, Hkv,
                                  Nt, Nk, d, block, 1.0 / math.sqrt(d) if scale is None else scale, ws, ws_bytes,
                                  handle), "fa_fwd_tree_fp8")
        return out, ls

    return _on(dev, stream, run)


def fa_cache_compact_fp8(k, v, k_scale, v_scale, kept, base=None, block: int = 64, k_out=None, v_out=None,
                         k_scale_out=None, v_scale_out=None, stream=None):
    """fa_cache_compact of a cache held in 8 bits: row base[b] + i of k_out,
    v_out [B, Hkv, Nk_out, d] becomes row base[b] + kept[b, h, i] of k, v where
    that entry is not negative, and a block that rows move to gets the greatest
    scale of the blocks they come from (with its own, where it holds rows before
    base).  kept: int32 [B, Hkv, M], or [B, M] for all heads.  Without outputs
    the cache is changed in place (the entries must then ascend, none below its
    place).  Returns (k_out, v_out, k_scale_out, v_scale_out)."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise TypeError("k must be a CUDA tensor")
    dev = k.device
    kp, ks = _view8("k", k, dev)
    B, Hkv, Nk, d = k.shape
    vp, vs = _view8("v", v, dev, k.shape)
    block = _block(block)
    outs = (k_out, v_out, k_scale_out, v_scale_out)
    if all(x is None for x in outs):
        k_out, v_out, k_scale_out, v_scale_out = k, v, k_scale, v_scale
    elif any(x is None for x in outs):
        raise ValueError("give all outputs or none")
    kop, kos = _view8("k_out", k_out, dev)
    Nout = k_out.shape[2]
    if k_out.shape != (B, Hkv, Nout, d):
        raise ValueError(f"k_out has shape {tuple(k_out.shape)}, expected ({B}, {Hkv}, Nk_out, {d})")
    vop, vos = _view8("v_out", v_out, dev, k_out.shape)
    ksp = _scale("k_scale", k_scale, B, Hkv, Nk, block, dev)
    vsp = _scale("v_scale", v_scale, B, Hkv, Nk, block, dev)
    kso = _scale("k_scale_out", k_scale_out, B, Hkv, Nout, block, dev)
    vso = _scale("v_scale_out", v_scale_out, B, Hkv, Nout, block, dev)
    if not isinstance(kept, torch.Tensor) or kept.dtype is not torch.int32 or kept.device != dev \
            or kept.dim() not in (2, 3):
        raise ValueError("kept must be an int32 tensor [B, Hkv, M] or [B, M]")
    st, M = kept.stride(), kept.shape[-1]
    if kept.shape not in ((B, Hkv, M), (B, M)) or (M > 1 and st[-1] != 1):
        raise ValueError(f"kept has shape {tuple(kept.shape)}, expected ({B}, {Hkv}, M) or ({B}, M), contiguous lists")
    bp = None if base is None else _plain("base", base, torch.int32, (B,), dev)

    def run(handle):
        _done(library().fa_cache_compact_fp8(kp, ks[0], vp, vs[0], ksp, vsp, kop, kos[0], vop, vos[0], kso, vso,
                                             kept.data_ptr(), st[0], st[1] if len(st) == 3 else 0, bp, B, Hkv, Nk, Nout,
                                             M, d, block, handle), "fa_cache_compact_fp8")
        return k_out, v_out, k_scale_out, v_scale_out

    return _on(dev, stream, run)


def _rows_of(name, t, B, Nt, dev, dtype):
    """[B, Nt] (any batch stride) or [Nt] (shared by the batch): pointer and batch stride."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev:
        raise ValueError(f"{name} must be a {dtype} tensor on {dev}")
    if t.shape not in ((B, Nt), (Nt,)) or (Nt > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({B}, {Nt}) or ({Nt},) with contiguous rows")
    return t.data_ptr(), t.stride(0) if t.dim() == 2 and B > 1 else 0


def _distributions(name, t, dev, shape=None):
    """fp32 [B, Nt, V] with contiguous V: pointer, batch and node strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.float32 or t.dim() != 3:
        raise TypeError(f"{name} must be an fp32 CUDA tensor [B, Nt, V]")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    B, Nt, V = t.shape
    st = t.stride()
    if V > 1 and st[2] != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), st[0] if B > 1 else 0, st[1] if Nt > 1 else 0


def fa_tree_verify(parents, tokens, target, draft, uniforms, accepted=None, counts=None, next_token=None, stream=None):
    """Drafted tokens verified against the target's probabilities.  parents and
    tokens (int32 [B, Nt] or [Nt]) are the tree, node 0 its root (decided, parent
    -1; anything else there marks padding); target and draft (fp32 [B, Nt, V])
    are the distributions at each node of the target and of the draft that its
    children were drawn from (``draft=None``: children chosen for certain);
    uniforms (fp32 [B, Nt] or [Nt], in [0, 1)) decide: a node's own whether it is
    accepted, node 0's the token that follows.  Returns (accepted int32 [B, Nt]:
    the nodes from the root on, -1 behind them, which is fa_cache_compact's list;
    counts int32 [B]; next_token int32 [B])."""
    tp, tb, tn = _distributions("target", target, None)
    B, Nt, V = target.shape
    dev = target.device
    dp, db, dn = (None, 0, 0) if draft is None else _distributions("draft", draft, dev, target.shape)
    pp, pb = _rows_of("parents", parents, B, Nt, dev, torch.int32)
    kp, kb = _rows_of("tokens", tokens, B, Nt, dev, torch.int32)
    up, ub = _rows_of("uniforms", uniforms, B, Nt, dev, torch.float32)

    def run(handle):
        acc = _empty((B, Nt), torch.int32, dev) if accepted is None else accepted
        num = _empty((B,), torch.int32, dev) if counts is None else counts
        nxt = _empty((B,), torch.int32, dev) if next_token is None else next_token
        _done(library().fa_tree_verify(pp, pb, kp, kb, tp, tb, tn, dp, db, dn, up, ub,
                                       _plain("accepted", acc, torch.int32, (B, Nt), dev),
                                       _plain("counts", num, torch.int32, (B,), dev),
                                       _plain("next_token", nxt, torch.int32, (B,), dev), B, Nt, V, handle),
              "fa_tree_verify")
        return acc, num, nxt

    return _on(dev, stream, run)
