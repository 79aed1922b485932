"""Paged grouped-query decode attention for GB300 (sm_103a).

Python face of the C ABI in include/gqa_decode.h: same operation names, torch
tensors in, argument marshalling only.  All computation runs in the library's
CUDA kernels; calling any op without the built library raises.

    kv_append(k_new, v_new, k_cache, v_cache, block_tables, context_lens)
    decode_attention(q, k_cache, v_cache, block_tables, context_lens) -> out
    verify_attention(q, k_cache, v_cache, block_tables, context_lens) -> out
    append_decode_attention(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens)
    append_verify_attention(...)  (kv_append fused into the attention launch)
    (every attention call takes window=W > 0 for local attention)
    kv_append_quant / decode_attention_quant / verify_attention_quant: the same
    over a one-byte (int8 or e4m3) cache with per-row fp32 scales
    accept_prefix(target_logits, draft_ids, context_lens=None) -> (accepted, next)
    accept_sampled(target_probs, draft_probs, draft_ids, uniforms,
                   context_lens=None) -> (accepted, next)
    accept_tree(target_logits, draft_ids, parents, context_lens=None)
        -> (accepted, next, path); then kv_compact(k_cache, v_cache, block_tables,
        context_lens, path, accepted) moves the accepted branch's cached rows
    kv="int4" on the _quant calls and kv_compact: a cache held in 4 bits
        (caches uint8 [NB,K,16,H/2], scales uint8 [NB,K,16,H/32])
    kv_append_slots(k_new, v_new, k_cache, v_cache, slots) / kv_gather_slots(...):
        packed rows [M,K,H] into and out of a cache of any kind, by slot
    plan_blocks(context_lens, new_lens, block_tables, held, free_ring, ring_state)
        -> lengths, blocks and slots of a step, made on the GPU
"""
from __future__ import annotations

import ctypes
import typing

import torch

from . import _lib
from ._lib import GqaError, Shape, Status, status_string  # noqa: F401

__all__ = ["kv_append", "kv_append_quant", "decode_attention", "verify_attention",
           "decode_attention_quant", "verify_attention_quant", "append_decode_attention_quant",
           "append_verify_attention_quant", "append_decode_attention",
           "append_verify_attention", "accept_prefix", "accept_sampled", "accept_tree",
           "kv_compact", "kv_append_slots", "kv_gather_slots", "plan_blocks", "BlockPlan",
           "attention_workspace_size", "reset_workspaces", "GqaError", "Status", "Shape"]


def reset_workspaces():
    """Drop the workspaces the binding caches per (device, stream); see
    _lib.reset_workspaces."""
    _lib.reset_workspaces()


def _status_arg(status):
    if status is None:
        return None
    _lib._need(status, "status", torch.int32)
    return _lib._ptr(status)


def kv_append(k_new, v_new, k_cache, v_cache, block_tables, context_lens, *, status=None,
              stream=None, pdl=False):
    """gqa_kv_append: k_new/v_new [B,T,K,H] -> caches [NB,16,K,H] at positions
    context_lens[b]-T+t.  Asynchronous on `stream` (default: current).
    pdl: launch with programmatic dependent launch (GQA_FLAG_PDL)."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _lib._need(t, n, ndim=4)
    _lib._need(block_tables, "block_tables", torch.int32, 2)
    _lib._need(context_lens, "context_lens", torch.int32, 1)
    shape = _lib.make_shape(k_new, k_cache, block_tables, None, heads_dim=3,
                            flags=_lib.FLAG_PDL if pdl else 0)
    rc = _lib.lib().gqa_kv_append(ctypes.byref(shape), _lib._ptr(k_new), _lib._ptr(v_new),
                                  _lib._ptr(k_cache), _lib._ptr(v_cache),
                                  _lib._ptr(block_tables), _lib._ptr(context_lens),
                                  _status_arg(status), _lib._stream(stream))
    _lib._check("gqa_kv_append", rc)


_BYTE_DTYPES = (torch.uint8, torch.int8, torch.float8_e4m3fn)


def _need_quant_cache(cache, scale, name):
    if not isinstance(cache, torch.Tensor) or cache.dtype not in _BYTE_DTYPES:
        raise ValueError(f"{name} must be a one-byte tensor (uint8 / int8 / float8_e4m3fn)")
    _lib._need(cache, name, ndim=4)
    _lib._need(scale, name + " scale", torch.float32, 3)
    NB, bs, K, _ = cache.shape
    if tuple(scale.shape) != (NB, K, bs):
        raise ValueError(f"{name} scale must be [{NB},{K},{bs}], got {tuple(scale.shape)}")


def kv_append_quant(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables,
                    context_lens, *, kv="int8", status=None, stream=None, pdl=False):
    """gqa_kv_append_quant: quantize k_new / v_new [B,T,K,H] (fp16 / bf16) row
    by row into one-byte caches [NB,16,K,H] and their scales fp32 [NB,K,16].
    kv="int4" (gqa_kv_append_fourbit): into 4-bit caches uint8 [NB,K,16,H/2] and
    their scales uint8 [NB,K,16,H/32]."""
    if kv == "int4":
        return _append4(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables,
                        context_lens, status, stream, pdl)
    _lib._need(k_new, "k_new", ndim=4)
    _lib._need(v_new, "v_new", k_new.dtype, 4)
    _need_quant_cache(k_cache, k_scale, "k_cache")
    _need_quant_cache(v_cache, v_scale, "v_cache")
    _lib._need(block_tables, "block_tables", torch.int32, 2)
    _lib._need(context_lens, "context_lens", torch.int32, 1)
    shape = _lib.make_shape(k_new, k_cache, block_tables, None, heads_dim=3,
                            flags=_lib.FLAG_PDL if pdl else 0, kv=kv)
    rc = _lib.lib().gqa_kv_append_quant(ctypes.byref(shape), _lib._ptr(k_new),
                                        _lib._ptr(v_new), _lib._ptr(k_cache),
                                        _lib._ptr(v_cache), _lib._ptr(k_scale),
                                        _lib._ptr(v_scale), _lib._ptr(block_tables),
                                        _lib._ptr(context_lens), _status_arg(status),
                                        _lib._stream(stream))
    _lib._check("gqa_kv_append_quant", rc)


def _shape_of_call(q, k_cache, block_tables, scale, window, kv, flags=0):
    """The shape of an attention call over a cache of kind kv."""
    if kv not in _lib.KV_DTYPES:
        raise ValueError(f"kv must be one of {sorted(_lib.KV_DTYPES)}, got {kv!r}")
    if kv != "int4":
        return _lib.make_shape(q, k_cache, block_tables, scale, window=window, flags=flags, kv=kv)
    B, T, N, _ = q.shape
    return _lib.make_shape4(q, k_cache, block_tables.shape[1], scale, B=B, T=T, N=N, flags=flags,
                            window=window)


def attention_engine(q, k_cache, block_tables, window=0, engine="auto", kv="same") -> str:
    """Which kernel serves an attention call of this shape: "warp" (the
    persistent mma.sync kernel), "direct" (mma.sync, one CTA per sequence and
    KV head), "tmem" (tcgen05 with tensor-memory accumulators) or "fourbit" (that
    of the 4-bit cache, kv="int4"); gqa_attention_engine.  Host logic only, for a
    call without a tree mask (a tree mask rules "direct" out)."""
    if engine not in _lib.ENGINES:
        raise ValueError(f"engine must be one of {sorted(_lib.ENGINES)}, got {engine!r}")
    shape = _shape_of_call(q, k_cache, block_tables, None, window, kv, _lib.ENGINES[engine])
    e = _lib.lib().gqa_attention_engine(ctypes.byref(shape))
    if e == 0:
        raise _lib.GqaError("gqa_attention_engine", _lib.Status.ERR_SHAPE)
    return _lib.ENGINE_NAMES[e]


def attention_workspace_size(q, k_cache, block_tables, scale=None, window=0, kv="same") -> int:
    """Workspace bytes of one attention call over a cache of kind kv ("same", "int8",
    "e4m3", "int4"), on the current GPU (a window never needs more than full attention
    of the same shape)."""
    return _lib.workspace_size(_shape_of_call(q, k_cache, block_tables, scale, window, kv))


def _attention(fn_name, q, k_cache, v_cache, block_tables, context_lens, out, scale,
               workspace, status, stream, pdl, early_kv, k_new=None, v_new=None, window=0,
               tree_mask=None, engine="auto"):
    _lib._need(q, "q", ndim=4)
    if engine not in _lib.ENGINES:
        raise ValueError(f"engine must be one of {sorted(_lib.ENGINES)}, got {engine!r}")
    if tree_mask is not None:
        _lib._need(tree_mask, "tree_mask", torch.int64, 2)  # uint64 bits, held as int64
        if tuple(tree_mask.shape) != tuple(q.shape[:2]):
            raise ValueError(f"tree_mask must be [B,T] = {tuple(q.shape[:2])}")
        fn_name = fn_name.replace("verify_attention", "tree_verify_attention")
    if k_new is not None:
        _lib._need(k_new, "k_new", q.dtype, 4)
        _lib._need(v_new, "v_new", q.dtype, 4)
    _lib._need(k_cache, "k_cache", q.dtype, 4)
    _lib._need(v_cache, "v_cache", q.dtype, 4)
    _lib._need(block_tables, "block_tables", torch.int32, 2)
    _lib._need(context_lens, "context_lens", torch.int32, 1)
    flags = ((_lib.FLAG_PDL if pdl else 0) | (_lib.FLAG_EARLY_KV if early_kv else 0)
             | _lib.ENGINES[engine])
    shape = _lib.make_shape(q, k_cache, block_tables, scale, flags=flags, window=window)
    if out is None:
        out = torch.empty_like(q)
    else:
        _lib._need(out, "out", q.dtype, 4)
    nbytes = _lib.workspace_size(shape)
    if workspace is None:
        workspace = _lib.get_workspace(nbytes, q.device, stream)
    else:
        _lib._need(workspace, "workspace", torch.uint8)
    L = _lib.lib()
    new = () if k_new is None else (_lib._ptr(k_new), _lib._ptr(v_new))
    mask = () if tree_mask is None else (_lib._ptr(tree_mask),)
    rc = getattr(L, fn_name)(ctypes.byref(shape), _lib._ptr(q), *new, _lib._ptr(k_cache),
                             _lib._ptr(v_cache), _lib._ptr(block_tables),
                             _lib._ptr(context_lens), *mask, _lib._ptr(out),
                             _lib._ptr(workspace), workspace.numel(), _status_arg(status),
                             _lib._stream(stream))
    _lib._check(fn_name, rc)
    return out


def decode_attention(q, k_cache, v_cache, block_tables, context_lens, *, out=None, scale=None,
                     workspace=None, status=None, stream=None, pdl=False, early_kv=False,
                     window=0, engine="auto"):
    """gqa_decode_attention (T == 1).  q [B,1,N,H] -> out [B,1,N,H].
    pdl / early_kv select GQA_FLAG_PDL / GQA_FLAG_EARLY_KV (see the C header);
    window > 0 is local attention over each query's last `window` positions;
    engine "warp" / "direct" / "tmem" forces the persistent mma.sync, the
    direct mma.sync or the tcgen05 kernel ("auto": by shape; GQA_FLAG_WARP_MMA
    / GQA_FLAG_DIRECT / GQA_FLAG_TENSOR_MEMORY)."""
    return _attention("gqa_decode_attention", q, k_cache, v_cache, block_tables, context_lens,
                      out, scale, workspace, status, stream, pdl, early_kv, window=window,
                      engine=engine)


def verify_attention(q, k_cache, v_cache, block_tables, context_lens, *, out=None, scale=None,
                     workspace=None, status=None, stream=None, pdl=False, early_kv=False,
                     window=0, tree_mask=None, engine="auto"):
    """gqa_verify_attention (T >= 1, causal among the T new tokens), or with
    tree_mask (int64 [B,T] holding the uint64 mask rows)
    gqa_tree_verify_attention."""
    return _attention("gqa_verify_attention", q, k_cache, v_cache, block_tables, context_lens,
                      out, scale, workspace, status, stream, pdl, early_kv, window=window,
                      tree_mask=tree_mask, engine=engine)


def append_decode_attention(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, *,
                            out=None, scale=None, workspace=None, status=None, stream=None,
                            pdl=False, early_kv=False, window=0, engine="auto"):
    """gqa_append_decode_attention: kv_append + decode_attention in one launch
    (T == 1).  Writes k_new/v_new into the caches and returns out."""
    return _attention("gqa_append_decode_attention", q, k_cache, v_cache, block_tables,
                      context_lens, out, scale, workspace, status, stream, pdl, early_kv,
                      k_new=k_new, v_new=v_new, window=window, engine=engine)


def append_verify_attention(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, *,
                            out=None, scale=None, workspace=None, status=None, stream=None,
                            pdl=False, early_kv=False, window=0, tree_mask=None,
                            engine="auto"):
    """gqa_append_verify_attention: kv_append + verify_attention in one launch
    (gqa_append_tree_verify_attention with tree_mask; with the tensor-memory
    kernel the append is a launch of its own just before)."""
    return _attention("gqa_append_verify_attention", q, k_cache, v_cache, block_tables,
                      context_lens, out, scale, workspace, status, stream, pdl, early_kv,
                      k_new=k_new, v_new=v_new, window=window, tree_mask=tree_mask,
                      engine=engine)


def _attention_quant(fn_name, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                     context_lens, out, scale, workspace, status, stream, pdl, early_kv, kv,
                     window=0, tree_mask=None):
    _lib._need(q, "q", ndim=4)
    if tree_mask is not None:
        _lib._need(tree_mask, "tree_mask", torch.int64, 2)  # uint64 bits, held as int64
        if tuple(tree_mask.shape) != tuple(q.shape[:2]):
            raise ValueError(f"tree_mask must be [B,T] = {tuple(q.shape[:2])}")
        fn_name = "gqa_tree_verify_attention_quant"
    _need_quant_cache(k_cache, k_scale, "k_cache")
    _need_quant_cache(v_cache, v_scale, "v_cache")
    _lib._need(block_tables, "block_tables", torch.int32, 2)
    _lib._need(context_lens, "context_lens", torch.int32, 1)
    flags = (_lib.FLAG_PDL if pdl else 0) | (_lib.FLAG_EARLY_KV if early_kv else 0)
    shape = _lib.make_shape(q, k_cache, block_tables, scale, flags=flags, window=window, kv=kv)
    if out is None:
        out = torch.empty_like(q)
    else:
        _lib._need(out, "out", q.dtype, 4)
    nbytes = _lib.workspace_size(shape)
    if workspace is None:
        workspace = _lib.get_workspace(nbytes, q.device, stream)
    else:
        _lib._need(workspace, "workspace", torch.uint8)
    mask = () if tree_mask is None else (_lib._ptr(tree_mask),)
    rc = getattr(_lib.lib(), fn_name)(ctypes.byref(shape), _lib._ptr(q), _lib._ptr(k_cache),
                                      _lib._ptr(v_cache), _lib._ptr(k_scale),
                                      _lib._ptr(v_scale), _lib._ptr(block_tables),
                                      _lib._ptr(context_lens), *mask, _lib._ptr(out),
                                      _lib._ptr(workspace), workspace.numel(),
                                      _status_arg(status), _lib._stream(stream))
    _lib._check(fn_name, rc)
    return out


def decode_attention_quant(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           *, kv="int8", out=None, scale=None, workspace=None, status=None,
                           stream=None, pdl=False, early_kv=False, window=0):
    """gqa_decode_attention_quant over a one-byte cache (kv = "int8" / "e4m3"),
    or gqa_attention_fourbit over a 4-bit one (kv = "int4", layouts as in
    kv_append_quant); window > 0 is local attention as in decode_attention."""
    if kv == "int4":
        return _attention4(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           None, None, out, scale, workspace, status, stream, pdl, early_kv,
                           window, None, True)
    return _attention_quant("gqa_decode_attention_quant", q, k_cache, v_cache, k_scale, v_scale,
                            block_tables, context_lens, out, scale, workspace, status, stream,
                            pdl, early_kv, kv, window)


def verify_attention_quant(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           *, kv="int8", out=None, scale=None, workspace=None, status=None,
                           stream=None, pdl=False, early_kv=False, window=0, tree_mask=None):
    """gqa_verify_attention_quant over a one-byte cache (kv = "int8" / "e4m3"), or
    gqa_attention_fourbit over a 4-bit one (kv = "int4");
    window > 0 is local attention and tree_mask (int64 [B,T] holding the uint64
    mask rows) tree verification, as in verify_attention
    (gqa_tree_verify_attention_quant)."""
    if kv == "int4":
        return _attention4(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           None, None, out, scale, workspace, status, stream, pdl, early_kv,
                           window, tree_mask, False)
    return _attention_quant("gqa_verify_attention_quant", q, k_cache, v_cache, k_scale, v_scale,
                            block_tables, context_lens, out, scale, workspace, status, stream,
                            pdl, early_kv, kv, window, tree_mask)


def _append_attention_quant(fn_name, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                            block_tables, context_lens, out, scale, workspace, status, stream,
                            pdl, early_kv, kv, window, tree_mask=None):
    if kv == "int4":
        return _attention4(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           k_new, v_new, out, scale, workspace, status, stream, pdl, early_kv,
                           window, tree_mask, "decode" in fn_name)
    if tree_mask is not None:
        raise ValueError('tree_mask needs kv="int4" here (one-byte caches: kv_append_quant, then '
                         "verify_attention_quant)")
    _lib._need(q, "q", ndim=4)
    _lib._need(k_new, "k_new", q.dtype, 4)
    _lib._need(v_new, "v_new", q.dtype, 4)
    _need_quant_cache(k_cache, k_scale, "k_cache")
    _need_quant_cache(v_cache, v_scale, "v_cache")
    _lib._need(block_tables, "block_tables", torch.int32, 2)
    _lib._need(context_lens, "context_lens", torch.int32, 1)
    flags = (_lib.FLAG_PDL if pdl else 0) | (_lib.FLAG_EARLY_KV if early_kv else 0)
    shape = _lib.make_shape(q, k_cache, block_tables, scale, flags=flags, window=window, kv=kv)
    if out is None:
        out = torch.empty_like(q)
    else:
        _lib._need(out, "out", q.dtype, 4)
    nbytes = _lib.workspace_size(shape)
    if workspace is None:
        workspace = _lib.get_workspace(nbytes, q.device, stream)
    else:
        _lib._need(workspace, "workspace", torch.uint8)
    P = _lib._ptr
    rc = getattr(_lib.lib(), fn_name)(ctypes.byref(shape), P(q), P(k_new), P(v_new),
                                      P(k_cache), P(v_cache), P(k_scale), P(v_scale),
                                      P(block_tables), P(context_lens), P(out), P(workspace),
                                      workspace.numel(), _status_arg(status),
                                      _lib._stream(stream))
    _lib._check(fn_name, rc)
    return out


def append_decode_attention_quant(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                  block_tables, context_lens, *, kv="int8", out=None,
                                  scale=None, workspace=None, status=None, stream=None,
                                  pdl=False, early_kv=False, window=0):
    """gqa_append_decode_attention_quant: kv_append_quant of the new token and
    decode attention over the one-byte cache in one call (two launches; the
    caches and their scales are written); kv = "int4" gives
    gqa_append_attention_fourbit."""
    return _append_attention_quant("gqa_append_decode_attention_quant", q, k_new, v_new,
                                   k_cache, v_cache, k_scale, v_scale, block_tables,
                                   context_lens, out, scale, workspace, status, stream, pdl,
                                   early_kv, kv, window)


def append_verify_attention_quant(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                  block_tables, context_lens, *, kv="int8", out=None,
                                  scale=None, workspace=None, status=None, stream=None,
                                  pdl=False, early_kv=False, window=0, tree_mask=None):
    """gqa_append_verify_attention_quant: the T new tokens appended to the
    one-byte cache and verify attention over it, in one call (two launches);
    kv = "int4" gives gqa_append_attention_fourbit, with tree_mask (as in
    verify_attention_quant) tree verification."""
    return _append_attention_quant("gqa_append_verify_attention_quant", q, k_new, v_new,
                                   k_cache, v_cache, k_scale, v_scale, block_tables,
                                   context_lens, out, scale, workspace, status, stream, pdl,
                                   early_kv, kv, window, tree_mask)


def accept_prefix(target_logits, draft_ids, context_lens=None, *, accepted=None,
                  next_token=None, status=None, stream=None, workspace=None, cluster=False):
    """gqa_accept_prefix.  target_logits fp32 [B,T,V], draft_ids int32 [B,T-1].
    Returns (accepted [B], next_token [B]); updates context_lens in place if given.
    workspace: uint8 device tensor of at least gqa_accept_workspace_size(B, T)
    bytes (default: one cached per stream); cluster=True passes no workspace
    (one thread-block cluster per sequence)."""
    _lib._need(target_logits, "target_logits", torch.float32, 3)
    B, T, V = target_logits.shape
    if T > 1:
        _lib._need(draft_ids, "draft_ids", torch.int32, 2)
    if context_lens is not None:
        _lib._need(context_lens, "context_lens", torch.int32, 1)
    dev = target_logits.device
    if accepted is None:
        accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=dev)
    L = _lib.lib()
    if cluster:
        workspace = None
    elif workspace is None:
        workspace = _lib.get_workspace(L.gqa_accept_workspace_size(B, T), dev, stream,
                                       kind="accept")
    else:
        _lib._need(workspace, "workspace", torch.uint8)
    rc = L.gqa_accept_prefix(B, T, V, _lib._ptr(target_logits),
                             _lib._ptr(draft_ids) if T > 1 else None,
                             _lib._ptr(accepted), _lib._ptr(next_token),
                             _lib._ptr(context_lens), _lib._ptr(workspace),
                             0 if workspace is None else workspace.numel(),
                             _status_arg(status), _lib._stream(stream))
    _lib._check("gqa_accept_prefix", rc)
    return accepted, next_token


def accept_tree(target_logits, draft_ids, parents, context_lens=None, *, accepted=None,
                next_token=None, path=None, status=None, stream=None, workspace=None,
                cluster=False):
    """gqa_accept_tree: greedy acceptance over a draft tree.  target_logits fp32
    [B,T,V] (row i: the target's prediction after node i's branch), draft_ids
    int32 [B,T-1] (node i's token at column i-1), parents int32 [B,T] (-1 for
    the root, then an index below the node's own).  Returns (accepted [B],
    next_token [B], path [B,T-1]: the accepted branch's nodes by depth, then
    -1); updates context_lens in place if given.  workspace / cluster as in
    accept_prefix."""
    _lib._need(target_logits, "target_logits", torch.float32, 3)
    B, T, V = target_logits.shape
    _lib._need(parents, "parents", torch.int32, 2)
    if tuple(parents.shape) != (B, T):
        raise ValueError(f"parents must be [{B},{T}], got {tuple(parents.shape)}")
    if T > 1:
        _lib._need(draft_ids, "draft_ids", torch.int32, 2)
        if tuple(draft_ids.shape) != (B, T - 1):
            raise ValueError(f"draft_ids must be [{B},{T - 1}], got {tuple(draft_ids.shape)}")
    if context_lens is not None:
        _lib._need(context_lens, "context_lens", torch.int32, 1)
    dev = target_logits.device
    if accepted is None:
        accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=dev)
    if path is None:
        path = torch.empty((B, max(T - 1, 0)), dtype=torch.int32, device=dev)
    else:
        _lib._need(path, "path", torch.int32, 2)
        if tuple(path.shape) != (B, max(T - 1, 0)):
            raise ValueError(f"path must be [{B},{max(T - 1, 0)}], got {tuple(path.shape)}")
    L = _lib.lib()
    if cluster:
        workspace = None
    elif workspace is None:
        workspace = _lib.get_workspace(L.gqa_accept_workspace_size(B, T), dev, stream,
                                       kind="accept")
    else:
        _lib._need(workspace, "workspace", torch.uint8)
    rc = L.gqa_accept_tree(B, T, V, _lib._ptr(target_logits),
                           _lib._ptr(draft_ids) if T > 1 else None, _lib._ptr(parents),
                           _lib._ptr(accepted), _lib._ptr(next_token),
                           _lib._ptr(path) if T > 1 else None, _lib._ptr(context_lens),
                           _lib._ptr(workspace), 0 if workspace is None else workspace.numel(),
                           _status_arg(status), _lib._stream(stream))
    _lib._check("gqa_accept_tree", rc)
    return accepted, next_token, path


def kv_compact(k_cache, v_cache, block_tables, context_lens, path, accepted, *, k_scale=None,
               v_scale=None, kv="same", status=None, stream=None, pdl=False):
    """gqa_kv_compact: after accept_tree, position base+j (j = 1..a, base =
    context_lens[b] - 1 - a, context_lens as accept_tree left them) takes the
    cached K and V rows of node path[b][j-1].  Caches [NB,16,K,H] in q's dtype
    (kv="same"), or one-byte caches with their scales fp32 [NB,K,16]
    (kv="int8" / "e4m3"), or 4-bit caches uint8 [NB,K,16,H/2] with theirs uint8
    [NB,K,16,H/32] (kv="int4").  The tree size T is path.shape[1] + 1."""
    if kv == "int4":
        return _compact4(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, path,
                         accepted, status, stream, pdl)
    if kv == "same":
        _lib._need(k_cache, "k_cache", ndim=4)
        _lib._need(v_cache, "v_cache", k_cache.dtype, 4)
        if k_cache.dtype not in _lib._DTYPES:
            raise ValueError(f"k_cache dtype {k_cache.dtype} unsupported (fp16 / bf16)")
        dtype = _lib._DTYPES[k_cache.dtype]
    else:
        _need_quant_cache(k_cache, k_scale, "k_cache")
        _need_quant_cache(v_cache, v_scale, "v_cache")
        dtype = 0
    _lib._need(block_tables, "block_tables", torch.int32, 2)
    _lib._need(context_lens, "context_lens", torch.int32, 1)
    _lib._need(path, "path", torch.int32, 2)
    _lib._need(accepted, "accepted", torch.int32, 1)
    NB, bs, K, H = k_cache.shape
    B = block_tables.shape[0]
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache must have the same shape")
    if context_lens.shape[0] != B or accepted.shape[0] != B or path.shape[0] != B:
        raise ValueError(f"context_lens, accepted and path must have {B} rows")
    shape = _lib.Shape(B=B, T=path.shape[1] + 1, N=K, K=K, H=H, block_size=bs, num_blocks=NB,
                       max_blocks_per_seq=block_tables.shape[1], dtype=dtype, scale=0.0,
                       flags=_lib.FLAG_PDL if pdl else 0, window=0,
                       kv_dtype=_lib.KV_DTYPES[kv])
    rc = _lib.lib().gqa_kv_compact(ctypes.byref(shape), _lib._ptr(k_cache), _lib._ptr(v_cache),
                                   _lib._ptr(k_scale), _lib._ptr(v_scale),
                                   _lib._ptr(block_tables), _lib._ptr(context_lens),
                                   _lib._ptr(path), _lib._ptr(accepted), _status_arg(status),
                                   _lib._stream(stream))
    _lib._check("gqa_kv_compact", rc)


def accept_sampled(target_probs, draft_probs, draft_ids, uniforms, context_lens=None, *,
                   accepted=None, next_token=None, status=None, stream=None):
    """gqa_accept_sampled.  target_probs fp32 [B,T,V], draft_probs fp32
    [B,T-1,V], draft_ids int32 [B,T-1], uniforms fp64 [B,T] in [0,1).
    Returns (accepted [B], next_token [B]); updates context_lens in place if given."""
    _lib._need(target_probs, "target_probs", torch.float32, 3)
    B, T, V = target_probs.shape
    _lib._need(uniforms, "uniforms", torch.float64, 2)
    if tuple(uniforms.shape) != (B, T):
        raise ValueError(f"uniforms must be [{B},{T}], got {tuple(uniforms.shape)}")
    if T > 1:
        _lib._need(draft_probs, "draft_probs", torch.float32, 3)
        _lib._need(draft_ids, "draft_ids", torch.int32, 2)
        if tuple(draft_probs.shape) != (B, T - 1, V) or tuple(draft_ids.shape) != (B, T - 1):
            raise ValueError("draft_probs must be [B,T-1,V] and draft_ids [B,T-1]")
    if context_lens is not None:
        _lib._need(context_lens, "context_lens", torch.int32, 1)
    dev = target_probs.device
    if accepted is None:
        accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=dev)
    rc = _lib.lib().gqa_accept_sampled(B, T, V, _lib._ptr(target_probs),
                                       _lib._ptr(draft_probs) if T > 1 else None,
                                       _lib._ptr(draft_ids) if T > 1 else None,
                                       _lib._ptr(uniforms), _lib._ptr(accepted),
                                       _lib._ptr(next_token), _lib._ptr(context_lens),
                                       _status_arg(status), _lib._stream(stream))
    _lib._check("gqa_accept_sampled", rc)
    return accepted, next_token


# ---- 4-bit cache, rows by slot, blocks of a step ------------------------------------------
# 4-bit attention, rows by slot and the planner are a few microseconds of GPU work at
# batch sizes where the host's part counts, so a combination of sizes and types is
# checked in full once: the checked C shape is kept under everything the checks looked
# at, and a later call of the same kind only makes sure that its tensors are contiguous
# and on one GPU.  (Rows by slot: the number of rows is one of the sizes.  The 4-bit
# append and compaction by block table check every call in full.)
_checked: dict = {}


def _remember(key, shape):
    if len(_checked) >= 4096:  # sizes keep changing (prompt lengths): start over
        _checked.clear()
    _checked[key] = shape = (shape, ctypes.byref(shape))
    return shape


def _need_cache4(cache, scale, name):
    _lib._need(cache, name, torch.uint8, 4)
    _lib._need(scale, name + " scale", torch.uint8, 4)
    NB, K, bs, half = cache.shape
    if tuple(scale.shape) != (NB, K, bs, half // 16):
        raise ValueError(f"{name} scale must be [{NB},{K},{bs},{half // 16}], got "
                         f"{tuple(scale.shape)}")


def _need_caches4(k_cache, v_cache, k_scale, v_scale):
    _need_cache4(k_cache, k_scale, "k_cache")
    _need_cache4(v_cache, v_scale, "v_cache")
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")


def _need_tables(block_tables, context_lens, B):
    _lib._need(block_tables, "block_tables", torch.int32, 2)
    _lib._need(context_lens, "context_lens", torch.int32, 1)
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError(f"block_tables and context_lens must have {B} rows")


def _need_rows4(x, name, B, T, K, dtype):
    _lib._need(x, name, dtype, 4)
    if tuple(x.shape[:3]) != (B, T, K):
        raise ValueError(f"{name} must be [{B},{T},{K},H], got {tuple(x.shape)}")


def _append4_shape(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   pdl):
    _need_caches4(k_cache, v_cache, k_scale, v_scale)
    _lib._need(k_new, "k_new", ndim=4)
    B, T = k_new.shape[:2]
    _need_rows4(k_new, "k_new", B, T, k_cache.shape[1], None)
    _need_rows4(v_new, "v_new", B, T, k_cache.shape[1], k_new.dtype)
    if v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must have the same shape")
    _need_tables(block_tables, context_lens, B)
    return _lib.make_shape4(k_new, k_cache, block_tables.shape[1], None, B=B, T=T,
                            N=k_cache.shape[1], flags=_lib.FLAG_PDL if pdl else 0)


def _append4(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
             status, stream, pdl):
    ts = (k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens)
    st = _status_arg(status)
    shape = _append4_shape(*ts, pdl)
    dev = _lib.one_device(*ts, status)
    with _lib.on_device(dev, stream) as s:
        rc = _lib.lib().gqa_kv_append_fourbit(ctypes.byref(shape), *(t.data_ptr() for t in ts),
                                              st, s.cuda_stream)
    _lib._check("gqa_kv_append_fourbit", rc)


def _attention4_shape(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables,
                      context_lens, scale, flags, window, tree_mask, decode):
    _lib._need(q, "q", ndim=4)
    B, T, N, H = q.shape
    if decode and T != 1:
        raise _lib.GqaError("gqa_attention_fourbit", _lib.Status.ERR_SHAPE)  # decode: T == 1
    _need_caches4(k_cache, v_cache, k_scale, v_scale)
    _need_tables(block_tables, context_lens, B)
    if k_new is not None:
        _need_rows4(k_new, "k_new", B, T, k_cache.shape[1], q.dtype)
        _need_rows4(v_new, "v_new", B, T, k_cache.shape[1], q.dtype)
        if k_new.shape[3] != H or v_new.shape[3] != H:
            raise ValueError(f"k_new and v_new must have head size {H}")
    if tree_mask is not None:
        _lib._need(tree_mask, "tree_mask", torch.int64, 2)  # uint64 bits, held as int64
        if tuple(tree_mask.shape) != (B, T):
            raise ValueError(f"tree_mask must be [B,T] = {(B, T)}")
    return _lib.make_shape4(q, k_cache, block_tables.shape[1], scale, B=B, T=T, N=N,
                            flags=flags, window=window)


def _attention4(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, k_new, v_new,
                out, scale, workspace, status, stream, pdl, early_kv, window, tree_mask, decode):
    scale, window = float(scale or 0.0), int(window)  # (a tensor's value, not the tensor)
    try:
        dev = q.get_device()
        key = (dev, decode, window, scale, pdl, early_kv, q.shape, q.dtype, k_cache.shape,
               k_cache.dtype, v_cache.shape, v_cache.dtype, k_scale.shape, k_scale.dtype,
               v_scale.shape, v_scale.dtype, block_tables.shape, block_tables.dtype,
               context_lens.shape, context_lens.dtype)
        fit = (q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
               and k_scale.is_contiguous() and v_scale.is_contiguous()
               and block_tables.is_contiguous() and context_lens.is_contiguous()
               and dev == k_cache.get_device() == v_cache.get_device() == k_scale.get_device()
               == v_scale.get_device() == block_tables.get_device() == context_lens.get_device())
        if k_new is not None:
            key += (k_new.shape, k_new.dtype, v_new.shape, v_new.dtype)
            fit = (fit and k_new.is_contiguous() and v_new.is_contiguous()
                   and dev == k_new.get_device() == v_new.get_device())
        if tree_mask is not None:
            key += ("tree", tree_mask.shape, tree_mask.dtype)
            fit = fit and tree_mask.is_contiguous() and dev == tree_mask.get_device()
        shape = _checked.get(key) if fit else None
    except (AttributeError, TypeError):
        key = shape = None
    if shape is None:
        flags = (_lib.FLAG_PDL if pdl else 0) | (_lib.FLAG_EARLY_KV if early_kv else 0)
        made = _attention4_shape(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                 block_tables, context_lens, scale, flags, window, tree_mask,
                                 decode)
        dev = _lib.one_device(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables,
                              context_lens, tree_mask).index
        with torch.cuda.device(dev):
            made.nbytes = _lib.workspace_size(made)
        shape = _remember(key, made)
    if stream is not None or dev != _lib.current_gpu():
        with _lib.on_device(torch.device("cuda", dev), stream):
            return _attention4(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                               k_new, v_new, out, scale, workspace, status, None, pdl, early_kv,
                               window, tree_mask, decode)
    if out is None:
        out = torch.empty_like(q)
    else:
        _lib._need(out, "out", q.dtype, 4)
        if out.shape != q.shape:
            raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(out.shape)}")
        _lib.one_device(q, out)
    st = None
    if status is not None:
        st = _status_arg(status)
        _lib.one_device(q, status)
    cs = _lib.raw_stream(dev)
    if workspace is None:
        workspace = _lib.get_workspace4(shape[0].nbytes, dev, cs)
    else:
        _lib._need(workspace, "workspace", torch.uint8)
        _lib.one_device(q, workspace)
    L = _lib.lib()
    mask = None if tree_mask is None else tree_mask.data_ptr()
    if k_new is None:
        rc = L.gqa_attention_fourbit(
            shape[1], q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), mask,
            out.data_ptr(), workspace.data_ptr(), workspace.numel(), st, cs)
    else:
        rc = L.gqa_append_attention_fourbit(
            shape[1], q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(),
            context_lens.data_ptr(), mask, out.data_ptr(), workspace.data_ptr(),
            workspace.numel(), st, cs)
    if rc:
        raise _lib.GqaError("gqa_attention_fourbit" if k_new is None
                            else "gqa_append_attention_fourbit", rc)
    return out


def _compact4(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, path, accepted,
              status, stream, pdl):
    _need_caches4(k_cache, v_cache, k_scale, v_scale)
    B = block_tables.shape[0]
    _need_tables(block_tables, context_lens, B)
    _lib._need(path, "path", torch.int32, 2)
    _lib._need(accepted, "accepted", torch.int32, 1)
    if accepted.shape[0] != B or path.shape[0] != B:
        raise ValueError(f"accepted and path must have {B} rows")
    NB, K, bs, half = k_cache.shape
    shape = _lib.Shape(B=B, T=path.shape[1] + 1, N=K, K=K, H=2 * half, block_size=bs,
                       num_blocks=NB, max_blocks_per_seq=block_tables.shape[1], dtype=0,
                       scale=0.0, flags=_lib.FLAG_PDL if pdl else 0, window=0,
                       kv_dtype=_lib.KV_DTYPES["int4"])
    ts = (k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, path, accepted)
    st = _status_arg(status)
    with _lib.on_device(_lib.one_device(*ts, status), stream) as s:
        rc = _lib.lib().gqa_kv_compact_fourbit(ctypes.byref(shape), *(t.data_ptr() for t in ts),
                                               st, s.cuda_stream)
    _lib._check("gqa_kv_compact_fourbit", rc)


# ---- rows by slot --------------------------------------------------------------------------
def _slots_shape(rows, k_cache, v_cache, k_scale, v_scale, kv, pdl):
    """Checks caches and packed rows [M,K,H] of a call by slot; its shape."""
    if kv not in _lib.KV_DTYPES:
        raise ValueError(f"kv must be one of {sorted(_lib.KV_DTYPES)}, got {kv!r}")
    if rows.dtype not in _lib._DTYPES:
        raise ValueError(f"dtype {rows.dtype} unsupported (fp16 / bf16)")
    H = rows.shape[2]
    flags = _lib.FLAG_PDL if pdl else 0
    if kv == "int4":
        _need_caches4(k_cache, v_cache, k_scale, v_scale)
        K = k_cache.shape[1]
        shape = _lib.make_shape4(rows, k_cache, 1, None, B=0, T=1, N=K, flags=flags)
    else:
        if kv == "same":
            _lib._need(k_cache, "k_cache", rows.dtype, 4)
            _lib._need(v_cache, "v_cache", rows.dtype, 4)
            if k_scale is not None or v_scale is not None:
                raise ValueError('kv="same" takes no scales')
        else:
            _need_quant_cache(k_cache, k_scale, "k_cache")
            _need_quant_cache(v_cache, v_scale, "v_cache")
        if k_cache.shape != v_cache.shape:
            raise ValueError("k_cache and v_cache must have the same shape")
        NB, bs, K, Hc = k_cache.shape
        if Hc != H:
            raise ValueError(f"head size mismatch: {H} vs {Hc}")
        shape = _lib.Shape(B=0, T=1, N=K, K=K, H=H, block_size=bs, num_blocks=NB,
                           max_blocks_per_seq=1, dtype=_lib._DTYPES[rows.dtype], scale=0.0,
                           flags=flags, window=0, kv_dtype=_lib.KV_DTYPES[kv])
    if rows.shape[1] != K:
        raise ValueError(f"rows have {rows.shape[1]} KV heads, the cache {K}")
    return shape


def _slots_call(k, v, k_cache, v_cache, k_scale, v_scale, slots, kv, pdl):
    """(checked shape, device index) of a call by slot; rows k and v [M,K,H]."""
    try:
        dev = k.get_device()
        key = (dev, kv, pdl, k.shape, k.dtype, v.shape, v.dtype, k_cache.shape, k_cache.dtype,
               v_cache.shape, v_cache.dtype, slots.shape, slots.dtype)
        fit = (k.is_contiguous() and v.is_contiguous() and k_cache.is_contiguous()
               and v_cache.is_contiguous() and slots.is_contiguous()
               and dev == v.get_device() == k_cache.get_device() == v_cache.get_device()
               == slots.get_device())
        if k_scale is not None or v_scale is not None:
            key += (k_scale.shape, k_scale.dtype, v_scale.shape, v_scale.dtype)
            fit = (fit and k_scale.is_contiguous() and v_scale.is_contiguous()
                   and dev == k_scale.get_device() == v_scale.get_device())
        shape = _checked.get(key) if fit else None
    except (AttributeError, TypeError):
        key = shape = None
    if shape is None:
        _lib._need(k, "k_new", ndim=3)
        _lib._need(v, "v_new", k.dtype, 3)
        if v.shape != k.shape:
            raise ValueError("k_new and v_new must have the same shape")
        _lib._need(slots, "slots", torch.int32, 1)
        if slots.shape[0] != k.shape[0]:
            raise ValueError(f"slots must have {k.shape[0]} entries, got {slots.shape[0]}")
        made = _slots_shape(k, k_cache, v_cache, k_scale, v_scale, kv, pdl)
        dev = _lib.one_device(k, v, k_cache, v_cache, k_scale, v_scale, slots).index
        shape = _remember(key, made)
    return shape, dev


def kv_append_slots(k_new, v_new, k_cache, v_cache, slots, *, k_scale=None, v_scale=None,
                    kv="same", status=None, stream=None, pdl=False):
    """gqa_kv_append_slots: packed rows k_new / v_new [M,K,H] (fp16 / bf16) into
    the slots slots[i] = block * 16 + row (int32 [M], -1: no slot) of a cache of
    any kind: kv="same" ([NB,16,K,H] in the rows' dtype, no scales), "int8" /
    "e4m3" (one byte, scales fp32 [NB,K,16]) or "int4" ([NB,K,16,H/2], scales
    uint8 [NB,K,16,H/32]).  The slots of one call must differ."""
    shape, dev = _slots_call(k_new, v_new, k_cache, v_cache, k_scale, v_scale, slots, kv, pdl)
    if stream is not None or dev != _lib.current_gpu():
        with _lib.on_device(torch.device("cuda", dev), stream):
            return kv_append_slots(k_new, v_new, k_cache, v_cache, slots, k_scale=k_scale,
                                   v_scale=v_scale, kv=kv, status=status, pdl=pdl)
    st = None
    if status is not None:
        st = _status_arg(status)
        _lib.one_device(k_new, status)
    rc = _lib.lib().gqa_kv_append_slots(
        shape[1], k_new.shape[0], k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
        None if v_scale is None else v_scale.data_ptr(), slots.data_ptr(), st,
        _lib.raw_stream(dev))
    if rc:
        raise _lib.GqaError("gqa_kv_append_slots", rc)


def kv_gather_slots(k_cache, v_cache, slots, *, k_scale=None, v_scale=None, kv="same",
                    dtype=None, k_out=None, v_out=None, status=None, stream=None, pdl=False):
    """gqa_kv_gather_slots: the cached rows of slots (int32 [M]; -1: zeros) as
    packed rows [M,K,H] in `dtype` (fp16 / bf16; default k_out's, or the cache's
    own for kv="same", else bf16).  Returns (k_out, v_out).  Caches and scales as
    in kv_append_slots."""
    if not (isinstance(k_cache, torch.Tensor) and isinstance(slots, torch.Tensor)):
        raise TypeError("k_cache and slots must be torch.Tensors")
    if k_cache.dim() != 4 or slots.dim() != 1:
        raise ValueError("k_cache must have 4 dims and slots 1")
    if not k_cache.is_cuda:
        raise ValueError("k_cache must be a CUDA tensor (the library has no CPU path)")
    if stream is not None or k_cache.get_device() != _lib.current_gpu():
        with _lib.on_device(k_cache.device, stream):
            return kv_gather_slots(k_cache, v_cache, slots, k_scale=k_scale, v_scale=v_scale,
                                   kv=kv, dtype=dtype, k_out=k_out, v_out=v_out, status=status,
                                   pdl=pdl)
    K, H = ((k_cache.shape[1], 2 * k_cache.shape[3]) if kv == "int4"
            else (k_cache.shape[2], k_cache.shape[3]))
    if dtype is None:
        dtype = (k_out.dtype if k_out is not None else k_cache.dtype if kv == "same"
                 else torch.bfloat16)
    want = (slots.shape[0], K, H)
    if k_out is None:
        k_out = torch.empty(want, dtype=dtype, device=k_cache.device)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    for t, n in ((k_out, "k_out"), (v_out, "v_out")):
        if tuple(t.shape) != want or t.dtype != dtype:
            raise ValueError(f"{n} must be {list(want)} of {dtype}, got {tuple(t.shape)}, {t.dtype}")
    shape, dev = _slots_call(k_out, v_out, k_cache, v_cache, k_scale, v_scale, slots, kv, pdl)
    st = None
    if status is not None:
        st = _status_arg(status)
        _lib.one_device(k_cache, status)
    rc = _lib.lib().gqa_kv_gather_slots(
        shape[1], want[0], k_cache.data_ptr(), v_cache.data_ptr(),
        None if k_scale is None else k_scale.data_ptr(),
        None if v_scale is None else v_scale.data_ptr(), slots.data_ptr(), k_out.data_ptr(),
        v_out.data_ptr(), st, _lib.raw_stream(dev))
    if rc:
        raise _lib.GqaError("gqa_kv_gather_slots", rc)
    return k_out, v_out


# ---- blocks of a step ------------------------------------------------------------------------
class BlockPlan(typing.NamedTuple):
    """What plan_blocks returns (block_tables and free_ring are updated in place)."""
    context_lens: torch.Tensor  # int32 [B] lengths with the new tokens
    held: torch.Tensor          # int32 [B] block-table entries in use
    ring_state: torch.Tensor    # int32 [2] head and count of the free ring
    cu_new: torch.Tensor        # int32 [B+1] first new token of each sequence
    slots: typing.Optional[torch.Tensor]      # int32 [max_tokens], -1 past the last
    positions: typing.Optional[torch.Tensor]  # int32 [max_tokens], -1 past the last


def _plan_check(ins, outs, max_tokens):
    """Checks plan_blocks' tensors (outs: (tensor or None, name, entries))."""
    for t, n, d in zip(ins, ("context_lens", "new_lens", "block_tables", "held", "free_ring",
                             "ring_state"), (1, 1, 2, 1, 1, 1)):
        _lib._need(t, n, torch.int32, d)
    B = ins[2].shape[0]
    if any(ins[i].shape[0] != B for i in (0, 1, 3)):
        raise ValueError(f"context_lens, new_lens and held must have {B} entries")
    if ins[5].shape[0] != 2:
        raise ValueError("ring_state must be [2]: head and count")
    for t, n, size in outs:
        if t is not None:
            _lib._need(t, n, torch.int32, 1)
            if t.shape[0] != size:
                raise ValueError(f"{n} must have {size} entries, got {t.shape[0]}")
    _lib.one_device(*ins, *(t for t, _, _ in outs))


def plan_blocks(context_lens, new_lens, block_tables, held, free_ring, ring_state, *,
                max_tokens=None, context_lens_out=None, held_out=None, ring_state_out=None,
                cu_new=None, slots=None, positions=None, in_place=False, status=None,
                stream=None, pdl=False) -> BlockPlan:
    """gqa_plan_blocks: grow every sequence by new_lens[b] tokens (int32 [B]; -1:
    finished, all its blocks go back), taking free block ids from the ring
    (free_ring int32 [num_blocks], ring_state int32 [2] = head, count) into
    block_tables [B, max_blocks] and returning those past ceil(length / 16);
    held int32 [B] counts each table's entries in use.  Slots and positions are
    made for up to max_tokens new tokens (default: the length of `slots`;
    neither given: no slot map).  The lengths, counts and state come back in new
    tensors, in the given ones, or with in_place=True in the inputs' own."""
    ins = (context_lens, new_lens, block_tables, held, free_ring, ring_state)
    if in_place:
        if not (context_lens_out is held_out is ring_state_out is None):
            raise ValueError("in_place=True takes no output tensors for what it updates")
        context_lens_out, held_out, ring_state_out = context_lens, held, ring_state
    if max_tokens is None:
        max_tokens = -1 if slots is None else slots.shape[0]
    if max_tokens > 2 ** 31 - 1:
        raise ValueError(f"max_tokens must be below 2**31, got {max_tokens}")
    if max_tokens < 0 and (slots is not None or positions is not None):
        raise ValueError("positions need slots or max_tokens")
    outs = (context_lens_out, held_out, ring_state_out, cu_new, slots, positions)
    try:
        dev = context_lens.get_device()
        key = ("plan", dev, max_tokens, context_lens.shape, context_lens.dtype, new_lens.shape,
               new_lens.dtype, block_tables.shape, block_tables.dtype, held.shape, held.dtype,
               free_ring.shape, free_ring.dtype, ring_state.shape, ring_state.dtype,
               *[None if t is None else (t.shape, t.dtype) for t in outs])
        fit = (context_lens.is_contiguous() and new_lens.is_contiguous()
               and block_tables.is_contiguous() and held.is_contiguous()
               and free_ring.is_contiguous() and ring_state.is_contiguous()
               and dev == new_lens.get_device() == block_tables.get_device()
               == held.get_device() == free_ring.get_device() == ring_state.get_device())
        for t in outs:
            if t is not None:
                fit = fit and t.is_contiguous() and dev == t.get_device()
        known = fit and key in _checked
    except (AttributeError, TypeError):
        key, known = None, False
    if not known:
        B = block_tables.shape[0] if isinstance(block_tables, torch.Tensor) else 0
        _plan_check(ins, ((context_lens_out, "context_lens_out", B), (held_out, "held_out", B),
                          (ring_state_out, "ring_state_out", 2), (cu_new, "cu_new", B + 1),
                          (slots, "slots", max_tokens), (positions, "positions", max_tokens)),
                    max_tokens)
        _remember(key, _lib.Shape())
        dev = context_lens.get_device()
    if stream is not None or dev != _lib.current_gpu():
        with _lib.on_device(torch.device("cuda", dev), stream):
            return plan_blocks(*ins, max_tokens=max_tokens,
                               context_lens_out=None if in_place else context_lens_out,
                               held_out=None if in_place else held_out,
                               ring_state_out=None if in_place else ring_state_out,
                               cu_new=cu_new, slots=slots, positions=positions,
                               in_place=in_place, status=status, pdl=pdl)
    B, mb = block_tables.shape
    if context_lens_out is None:
        context_lens_out = torch.empty_like(context_lens)
    if held_out is None:
        held_out = torch.empty_like(held)
    if ring_state_out is None:
        ring_state_out = torch.empty_like(ring_state)
    if cu_new is None:
        cu_new = context_lens.new_empty(B + 1)
    if max_tokens >= 0:
        if slots is None:
            slots = context_lens.new_empty(max_tokens)
        if positions is None:
            positions = context_lens.new_empty(max_tokens)
    st = None
    if status is not None:
        st = _status_arg(status)
        _lib.one_device(context_lens, status)
    some = max_tokens > 0
    rc = _lib.lib().gqa_plan_blocks(
        B, mb, free_ring.shape[0], max_tokens, context_lens.data_ptr(), new_lens.data_ptr(),
        held.data_ptr(), ring_state.data_ptr(), free_ring.data_ptr(), block_tables.data_ptr(),
        context_lens_out.data_ptr(), held_out.data_ptr(), ring_state_out.data_ptr(),
        cu_new.data_ptr(), slots.data_ptr() if some else None,
        positions.data_ptr() if some else None, _lib.FLAG_PDL if pdl else 0, st,
        _lib.raw_stream(dev))
    if rc:
        raise _lib.GqaError("gqa_plan_blocks", rc)
    return BlockPlan(context_lens_out, held_out, ring_state_out, cu_new, slots, positions)
