"""Decode-step operators over a paged KV cache (see include/vts.h).

    tree_attention(q, k_cache, v_cache, page_table, seq_lens, ...)  -> (out, lse | None)
    attention_weight_add(weights, q, k_cache, page_table, seq_lens, lse, ...) -> weights
    evict_cache(weights, k_cache, v_cache, page_table, seq_lens, keep, k_out, v_out,
                out_page_table, ...)                       -> (kept, seq_lens, weights)
    verify_draft(target_probs, draft_tokens, uniforms, ...) -> (path, count, next_token)
    tree_mask_from_parents(parents)                         -> tree_mask

A cache is a 4-D tensor ``[num_pages, page_size, kv_heads, head_dim]`` of any
strides that are multiples of 8 elements (so a cache laid out heads first is
passed as a permuted view), bfloat16 or float16; ``tree_attention`` also takes
microscaled caches of uint8 rows with their scales (``varlen_top_select_amd.cache``).
Lengths count the drafted tokens, as ``next_n`` does in ``topk_varlen``.  The operators
serve decoding and have no derivatives: their outputs carry no gradient, also of
inputs that require one.

Without ``workspace`` the calls share one per device and stream, made at the first
eager call and held until the process ends, also where a larger shape has
replaced it: graphs captured with it stay valid.  Graphs captured on one stream
share that stream's workspace, so replay them one after another, or give each
its own: ``torch.zeros`` of the bytes that ``tree_attention_workspace_bytes`` or
``verify_draft_workspace_bytes`` says.
"""
from __future__ import annotations

import functools
import math
import struct

import torch

from . import _DTYPE, _check, _default_workspace, library

__all__ = ["tree_attention", "attention_weight_add", "evict_cache", "verify_draft",
           "tree_mask_from_parents", "tree_attention_workspace_bytes",
           "verify_draft_workspace_bytes"]

_CACHE = struct.Struct("@QQqqqqqqQqqQqiiiii4x")  # vts_paged_cache
_STRIDES = struct.Struct("@qqq")
_SCALES = struct.Struct("@QQqqqqqqi4x")  # vts_microscales
MAX_DRAFT = 64


# The checks below run before every launch; sizes and devices are compared as
# plain numbers, which costs a fraction of comparing torch.device objects.


# the current stream's handle of a device, without making a Stream object of it
_current = getattr(torch._C, "_cuda_getCurrentRawStream",
                   lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(stream, index, call):
    """call(stream pointer) with device `index` and, where one is given, `stream`
    current, so that what the call allocates belongs to the stream it runs on."""
    if stream is None:
        if index == torch.cuda.current_device():
            return call(_current(index))
        with torch.cuda.device(index):
            return call(_current(index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _workspace(workspace, need, device, sp):
    if workspace is None:
        return _default_workspace(need, device, sp, "decode")
    if (not isinstance(workspace, torch.Tensor) or workspace.device != device
            or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


@functools.lru_cache(maxsize=256)
def tree_attention_workspace_bytes(batch, draft, heads, kv_heads, head_dim, top_k=0, microscaled=False):
    """Bytes of a workspace (zeroed once) for tree_attention calls of this shape, over
    16-bit or (8 and 4 bits) microscaled caches."""
    lib = library()
    f = (lib.vts_tree_attention_microscaled_workspace_bytes if microscaled
         else lib.vts_tree_attention_workspace_bytes)
    return f(batch, draft, heads, kv_heads, head_dim, top_k)


@functools.lru_cache(maxsize=256)
def verify_draft_workspace_bytes(batch, vocab):
    """Bytes of a workspace (zeroed once) for verify_draft calls of this shape."""
    return library().vts_verify_draft_workspace_bytes(batch, vocab)


def _steps(t, low=7):
    """The strides of a 4-D tensor's first three dimensions (0 where a dimension has one
    element, whose stride means nothing), or None where its rows are no aligned vectors
    of low + 1 elements."""
    a, b, c, d = t.stride()
    if (a | b | c) & low or d != 1:
        n = t.shape
        a, b, c = a if n[0] > 1 else 0, b if n[1] > 1 else 0, c if n[2] > 1 else 0
        if (a | b | c) & low or d != 1:
            return None
    return a, b, c


def _row_step(t, rows):
    """The stride between a table's contiguous rows, or None."""
    if t.stride(1) != 1 and t.shape[1] > 1:
        return None
    return t.stride(0) if rows > 1 else t.shape[1]


def _cache(name, t, like=None):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a 4-D tensor [pages, page_size, kv_heads, head_dim]")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float16:
        raise ValueError(f"{name} dtype must be bfloat16 or float16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must have the other cache's dtype and device")
    steps = _steps(t)
    if steps is None or t.data_ptr() & 15:
        raise ValueError(f"{name} rows must be contiguous, 16-byte aligned, with strides that "
                         "are multiples of 8 elements")
    return steps


def _tensor(name, t, dtype, shape, index):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{index}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {shape}")
    return t


def _table(name, t, batch, index):
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.get_device() != index
            or t.dim() != 2 or t.shape[0] != batch or t.shape[1] < 1
            or (step := _row_step(t, batch)) is None):
        raise ValueError(f"{name} must be an int32 tensor of {batch} contiguous rows on cuda:{index}")
    return step


def _rows(name, t, low, index):
    """The strides of a microscaled cache's tensor, or of its scales."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8 or t.get_device() != index or t.dim() != 4:
        raise ValueError(f"{name} must be a 4-D uint8 tensor on cuda:{index}")
    a, b, c, d = t.stride()
    if ((a | b | c | t.data_ptr()) & low) == 0 and d == 1:
        return a, b, c
    steps = _steps(t, low)
    if steps is None or t.data_ptr() & low:
        raise ValueError(f"{name} rows must be contiguous, with an address and strides that are multiples "
                         f"of {low + 1} bytes")
    return steps


def _micro(k_cache, v_cache, k_scales, v_scales):
    """(the caches' strides, vts_microscales as bytes, device index, head_dim)"""
    if k_scales is None or v_scales is None:
        raise ValueError("k_scales and v_scales must be given together")
    if not isinstance(k_cache, torch.Tensor) or not k_cache.is_cuda:
        raise ValueError("k_cache must be on the GPU")
    index = k_cache.get_device()
    ks, vs = _rows("k_cache", k_cache, 15, index), _rows("v_cache", v_cache, 15, index)
    if not isinstance(k_scales, torch.Tensor) or k_scales.dim() != 4:
        raise ValueError("k_scales must be a 4-D tensor [pages, page_size, kv_heads, head_dim / 32]")
    pages, page_size, kv_heads, row = shape = k_cache.shape
    blocks = k_scales.shape[3]
    if blocks != 4 and blocks != 2:
        raise ValueError("k_scales must be of head_dim 64 or 128, a scale to 32 elements")
    kss, vss = _rows("k_scales", k_scales, blocks - 1, index), _rows("v_scales", v_scales, blocks - 1, index)
    scales = (pages, page_size, kv_heads, blocks)
    if v_cache.shape != shape or k_scales.shape != scales or v_scales.shape != scales or row not in (
            32 * blocks, 16 * blocks):
        raise ValueError("a microscaled cache's rows must be head_dim (8 bits) or head_dim / 2 (4 bits) bytes, its "
                         "scales [pages, page_size, kv_heads, head_dim / 32], and V's tensors must have the shapes "
                         "of K's")
    packed = _SCALES.pack(k_scales.data_ptr(), v_scales.data_ptr(), *kss, *vss, row // (4 * blocks))
    return ks, vs, packed, index, 32 * blocks


def _paged_micro(k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, dtype):
    """_paged of a microscaled cache, and its vts_microscales as bytes"""
    ks, vs, scales, index, head_dim = _micro(k_cache, v_cache, k_scales, v_scales)
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("q dtype must be bfloat16 or float16")
    pages, page_size, kv_heads, _ = k_cache.shape
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be a 1-D tensor")
    batch = seq_lens.shape[0]
    _tensor("seq_lens", seq_lens, torch.int32, (batch,), index)
    stride = _table("page_table", page_table, batch, index)
    packed = _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), *ks, *vs, page_table.data_ptr(), stride,
                         page_table.shape[1], seq_lens.data_ptr(), pages, page_size, kv_heads,
                         head_dim, batch, _DTYPE[dtype])
    return packed, scales, index, batch, kv_heads, head_dim


def _paged(k_cache, v_cache, page_table, seq_lens):
    """(vts_paged_cache as bytes, device index, batch, kv_heads, head_dim)"""
    ks = _cache("k_cache", k_cache)
    index = k_cache.get_device()
    pages, page_size, kv_heads, head_dim = k_cache.shape
    if v_cache is None:
        vs, vp = ks, 0
    else:
        vs, vp = _cache("v_cache", v_cache, k_cache), v_cache.data_ptr()
        if v_cache.shape != k_cache.shape:
            raise ValueError("v_cache must have the shape of k_cache")
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be a 1-D tensor")
    batch = seq_lens.shape[0]
    _tensor("seq_lens", seq_lens, torch.int32, (batch,), index)
    stride = _table("page_table", page_table, batch, index)
    packed = _CACHE.pack(k_cache.data_ptr(), vp, *ks, *vs, page_table.data_ptr(), stride,
                         page_table.shape[1], seq_lens.data_ptr(), pages, page_size, kv_heads,
                         head_dim, batch, _DTYPE[k_cache.dtype])
    return packed, index, batch, kv_heads, head_dim


def _meets(out, t):
    """Whether the contiguous `out` has memory in common with the rows of the 4-D t."""
    if not out.numel() or not t.numel():
        return False
    e = t.element_size()
    lo, hi = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    row = t.shape[3] * e
    dims = sorted(((n, s * e) for n, s in zip(t.shape[:3], t.stride()) if n > 1 and s), key=lambda d: -d[1])

    def within(at, i):  # some row of t's last dimensions i.. that begin at `at`
        if i == len(dims):
            return at < hi and at + row > lo
        n, s = dims[i]
        reach = row + sum((m - 1) * d for m, d in dims[i + 1:])
        first = max(0, (lo - at - reach) // s + 1)  # the steps that end past lo
        last = min(n - 1, (hi - at - 1) // s)       # those that begin before hi
        if first <= last and at + last * s >= lo:
            return True  # a row begins in there
        return any(within(at + j * s, i + 1) for j in range(first, last + 1))

    return within(t.data_ptr(), 0)


def _query(q, dtype, batch, kv_heads, head_dim, index):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D tensor [batch, draft, heads, head_dim]")
    n, draft, heads, dim = q.shape
    if q.dtype is not dtype or q.get_device() != index or n != batch or dim != head_dim:
        raise ValueError("q must have the cache's dtype, device and head_dim, and the batch of "
                         "seq_lens")
    if not 1 <= draft <= MAX_DRAFT:
        raise ValueError(f"q must have 1..{MAX_DRAFT} drafted tokens a request")
    if heads < kv_heads or heads % kv_heads:
        raise ValueError("the query heads must be a multiple of the KV heads")
    steps = _steps(q)
    if steps is None or q.data_ptr() & 15:
        raise ValueError("q rows must be contiguous, 16-byte aligned, with strides that are "
                         "multiples of 8 elements")
    return draft, heads, _STRIDES.pack(*steps)


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   page_table: torch.Tensor, seq_lens: torch.Tensor, *,
                   tree_mask: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                   scale: float | None = None, out: torch.Tensor | None = None,
                   return_lse: bool = False, workspace: torch.Tensor | None = None, stream=None,
                   k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
    """Attention of q[batch, draft, heads, head_dim] over each request's cached
    prefix (or the listed ``slots``) and the drafted tokens that ``tree_mask``
    names (vts_tree_attention in include/vts.h).  Returns the outputs, in ``out`` if
    given, which must not overlap q or the caches, and the rows' log-sum-exp or None.
    With ``k_scales`` and ``v_scales`` the caches are microscaled: uint8 rows of
    head_dim (8 bits) or head_dim / 2 bytes (4 bits), and uint8 scales [pages, page_size,
    kv_heads, head_dim / 32]; q is then bfloat16 or float16."""
    micro = k_scales is not None or v_scales is not None
    if micro:
        if not isinstance(q, torch.Tensor):
            raise ValueError("q must be a 4-D tensor [batch, draft, heads, head_dim]")
        cache, scales, index, batch, kv_heads, head_dim = _paged_micro(
            k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, q.dtype)
    else:
        cache, index, batch, kv_heads, head_dim = _paged(k_cache, v_cache, page_table, seq_lens)
    draft, heads, q_strides = _query(q, q.dtype if micro else k_cache.dtype, batch, kv_heads, head_dim, index)
    mask_ptr = slots_ptr = None
    top_k = 0
    if tree_mask is not None:
        mask_ptr = _tensor("tree_mask", tree_mask, torch.int64, (batch, draft), index).data_ptr()
    if slots is not None:
        if not isinstance(slots, torch.Tensor) or slots.numel() == 0 and batch:
            raise ValueError("slots must be a non-empty tensor")
        top_k = slots.shape[-1]
        shape = (batch, draft, top_k) if slots.dim() == 3 else (batch * draft, top_k)
        slots_ptr = _tensor("slots", slots, torch.int32, shape, index).data_ptr()
    if out is not None:
        _tensor("out", out, q.dtype, (batch, draft, heads, head_dim), index)
        if any(_meets(out, t) for t in (q, k_cache, v_cache, k_scales, v_scales) if t is not None):
            raise ValueError("out must not overlap q or the caches")
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    lib, device = library(), q.device

    def call(sp):
        o = torch.empty((batch, draft, heads, head_dim), dtype=q.dtype,
                        device=device) if out is None else out
        lse = torch.empty((batch, draft, heads), dtype=torch.float32,
                          device=device) if return_lse else None
        ws = _workspace(workspace, tree_attention_workspace_bytes(batch, draft, heads, kv_heads, head_dim,
                                                                  top_k, micro), device, sp)
        if micro:
            _check("vts_tree_attention_microscaled", lib.vts_tree_attention_microscaled(
                cache, scales, q.data_ptr(), q_strides, draft, heads, mask_ptr, slots_ptr, top_k, scale,
                o.data_ptr(), lse.data_ptr() if return_lse else None, ws.data_ptr(),
                ws.numel() * ws.element_size(), sp))
            return o, lse
        _check("vts_tree_attention", lib.vts_tree_attention(
            cache, q.data_ptr(), q_strides, draft, heads, mask_ptr, slots_ptr, top_k, scale,
            o.data_ptr(), lse.data_ptr() if return_lse else None, ws.data_ptr(),
            ws.numel() * ws.element_size(), sp))
        return o, lse

    return _run(stream, index, call)


def _weights(name, w, batch, kv_heads, index):
    if (not isinstance(w, torch.Tensor) or w.dtype is not torch.float32 or w.get_device() != index
            or w.dim() != 3 or w.shape[0] != batch or w.shape[1] != kv_heads
            or (w.stride(2) != 1 and w.shape[2] > 1)):
        raise ValueError(f"{name} must be a float32 tensor [{batch}, {kv_heads}, width] with "
                         f"contiguous rows on cuda:{index}")
    return w.stride(0), w.stride(1), w.shape[2]


def attention_weight_add(weights: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                         page_table: torch.Tensor, seq_lens: torch.Tensor, lse: torch.Tensor, *,
                         tree_mask: torch.Tensor | None = None,
                         row_keep: torch.Tensor | None = None, scale: float | None = None,
                         stream=None) -> torch.Tensor:
    """weights[batch, kv_heads, width] += the attention weight that each cached
    entry got from the rows of q that ``row_keep`` counts; lse as
    tree_attention returned it (vts_attention_weight_add in include/vts.h)."""
    cache, index, batch, kv_heads, head_dim = _paged(k_cache, None, page_table, seq_lens)
    draft, heads, q_strides = _query(q, k_cache.dtype, batch, kv_heads, head_dim, index)
    wb, wh, width = _weights("weights", weights, batch, kv_heads, index)
    if (batch > 1 and wb < width) or (kv_heads > 1 and wh < width):
        raise ValueError("weights rows must not overlap")
    _tensor("lse", lse, torch.float32, (batch, draft, heads), index)
    mask_ptr = keep_ptr = None
    if tree_mask is not None:
        mask_ptr = _tensor("tree_mask", tree_mask, torch.int64, (batch, draft), index).data_ptr()
    if row_keep is not None:
        if not isinstance(row_keep, torch.Tensor) or row_keep.dtype not in (torch.bool, torch.uint8):
            raise ValueError("row_keep must be a bool or uint8 tensor")
        keep_ptr = _tensor("row_keep", row_keep, row_keep.dtype, (batch, draft), index).data_ptr()
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    lib = library()

    def call(sp):
        _check("vts_attention_weight_add", lib.vts_attention_weight_add(
            cache, q.data_ptr(), q_strides, draft, heads, mask_ptr, lse.data_ptr(), keep_ptr,
            scale, weights.data_ptr(), wb, wh, width, sp))
        return weights

    return _run(stream, index, call)


def evict_cache(weights: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                page_table: torch.Tensor, seq_lens: torch.Tensor, keep: int,
                k_out: torch.Tensor, v_out: torch.Tensor, out_page_table: torch.Tensor, *,
                sinks: int = 0, recent: int = 0, stream=None):
    """Keeps at most ``keep`` entries per request and KV head, the first
    ``sinks``, the last ``recent`` and the heaviest of the rest, and moves them
    to the pages of ``out_page_table`` in ``k_out`` and ``v_out`` (vts_evict_cache in
    include/vts.h).  Returns the kept positions [batch, kv_heads, keep] (-1 in
    unused entries), the new lengths [batch] and the kept weights."""
    cache, index, batch, kv_heads, head_dim = _paged(k_cache, v_cache, page_table, seq_lens)
    wb, wh, width = _weights("weights", weights, batch, kv_heads, index)
    if keep < 1 or sinks < 0 or recent < 0 or sinks + recent > keep:
        raise ValueError("keep must be at least 1 and at least sinks + recent")
    ko, vo = _cache("k_out", k_out, k_cache), _cache("v_out", v_out, k_cache)
    if k_out.shape[1:] != k_cache.shape[1:] or v_out.shape != k_out.shape:
        raise ValueError("k_out and v_out must be caches of the same page_size, heads and head_dim")
    stride = _table("out_page_table", out_page_table, batch, index)
    if out_page_table.shape[1] * k_cache.shape[1] < keep:
        raise ValueError("out_page_table must have pages for `keep` entries")
    lib, device = library(), k_cache.device

    def call(sp):
        kept = torch.empty((batch, kv_heads, keep), dtype=torch.int32, device=device)
        lens = torch.empty((batch,), dtype=torch.int32, device=device)
        w = torch.empty((batch, kv_heads, keep), dtype=torch.float32, device=device)
        _check("vts_evict_cache", lib.vts_evict_cache(
            cache, weights.data_ptr(), wb, wh, width, keep, sinks, recent, k_out.data_ptr(),
            _STRIDES.pack(*ko), v_out.data_ptr(), _STRIDES.pack(*vo), k_out.shape[0],
            out_page_table.data_ptr(), stride, out_page_table.shape[1], kept.data_ptr(),
            lens.data_ptr(), w.data_ptr(), sp))
        return kept, lens, w

    return _run(stream, index, call)


def verify_draft(target_probs: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor, *,
                 draft_probs: torch.Tensor | None = None, parents: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """Verifies draft_tokens[batch, draft] (a chain, or a tree given by
    ``parents``) against target_probs[batch, draft + 1, vocab] with the random
    numbers uniforms[batch, draft + 1] in [0, 1) (vts_verify_draft in
    include/vts.h).  Tokens of -1 pad a request that has fewer.  Returns the
    accepted nodes [batch, draft] (-1 past them), their number [batch] and the
    next token [batch], all int32."""
    if not isinstance(target_probs, torch.Tensor) or target_probs.dim() != 3:
        raise ValueError("target_probs must be a 3-D tensor [batch, draft + 1, vocab]")
    if target_probs.dtype not in _DTYPE:
        raise ValueError("target_probs dtype must be float32, bfloat16 or float16")
    if not target_probs.is_cuda:
        raise ValueError("target_probs must be on the GPU")
    index = target_probs.get_device()
    batch, draft, vocab = target_probs.shape
    draft -= 1
    if not 1 <= draft <= MAX_DRAFT or vocab < 1:
        raise ValueError(f"target_probs must have 2..{MAX_DRAFT + 1} rows a request, not empty")
    if target_probs.stride(2) != 1 and vocab > 1:
        raise ValueError("target_probs rows must be contiguous")
    _tensor("draft_tokens", draft_tokens, torch.int32, (batch, draft), index)
    _tensor("uniforms", uniforms, torch.float32, (batch, draft + 1), index)
    q_ptr = parents_ptr = None
    qb = qr = 0
    if draft_probs is not None:
        if (not isinstance(draft_probs, torch.Tensor) or draft_probs.dtype is not target_probs.dtype
                or draft_probs.get_device() != index or draft_probs.shape != (batch, draft, vocab)
                or (draft_probs.stride(2) != 1 and vocab > 1)):
            raise ValueError("draft_probs must be a tensor [batch, draft, vocab] with contiguous "
                             "rows, of target_probs' dtype and device")
        q_ptr = draft_probs.data_ptr()
        qb, qr = draft_probs.stride(0), draft_probs.stride(1)
    if parents is not None:
        parents_ptr = _tensor("parents", parents, torch.int32, (batch, draft), index).data_ptr()
    lib, device = library(), target_probs.device

    def call(sp):
        path = torch.empty((batch, draft), dtype=torch.int32, device=device)
        count = torch.empty((batch,), dtype=torch.int32, device=device)
        token = torch.empty((batch,), dtype=torch.int32, device=device)
        ws = _workspace(workspace, verify_draft_workspace_bytes(batch, vocab), device, sp)
        _check("vts_verify_draft", lib.vts_verify_draft(
            target_probs.data_ptr(), _DTYPE[target_probs.dtype], target_probs.stride(0),
            target_probs.stride(1), q_ptr, qb, qr, draft_tokens.data_ptr(), parents_ptr,
            uniforms.data_ptr(), batch, draft, vocab, path.data_ptr(), count.data_ptr(),
            token.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), sp))
        return path, count, token

    return _run(stream, index, call)


def tree_mask_from_parents(parents: torch.Tensor) -> torch.Tensor:
    """tree_mask[batch, draft] of trees given by parents[batch, draft] (-1: hangs
    from the context): each node sees its ancestors and itself.  A node whose
    parent does not exist, outside [-1, draft), sees itself alone."""
    if parents.dim() != 2 or parents.shape[1] > MAX_DRAFT:
        raise ValueError(f"parents must be a 2-D tensor of at most {MAX_DRAFT} columns")
    draft = parents.shape[1]
    bits = (1 << torch.arange(draft, dtype=torch.int64, device=parents.device)).expand_as(parents)
    jump = parents.long()
    jump = torch.where(jump < draft, jump, -1)  # (an index past the row would end the process on a GPU)
    for _ in range(max(1, draft - 1).bit_length()):  # bits cover twice as many generations each time
        up = jump.clamp(min=0)
        bits = torch.where(jump >= 0, bits | bits.gather(1, up), bits)
        jump = torch.where(jump >= 0, jump.gather(1, up), jump)
    return bits.contiguous()


def declare(lib):
    """Argument types of the C entry points."""
    import ctypes

    vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float)
    lib.vts_tree_attention_workspace_bytes.restype = sz
    lib.vts_tree_attention_workspace_bytes.argtypes = [i32] * 6
    lib.vts_tree_attention.restype = ctypes.c_int
    lib.vts_tree_attention.argtypes = [vp, vp, vp, i32, i32, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    lib.vts_tree_attention_microscaled_workspace_bytes.restype = sz
    lib.vts_tree_attention_microscaled_workspace_bytes.argtypes = [i32] * 6
    lib.vts_tree_attention_microscaled.restype = ctypes.c_int
    lib.vts_tree_attention_microscaled.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, i32, f32, vp, vp, vp,
                                                   sz, vp]
    lib.vts_attention_weight_add.restype = ctypes.c_int
    lib.vts_attention_weight_add.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, f32, vp, i64, i64,
                                             i64, vp]
    lib.vts_evict_cache.restype = ctypes.c_int
    lib.vts_evict_cache.argtypes = [vp, vp, i64, i64, i64, i32, i32, i32, vp, vp, vp, vp, i64, vp,
                                    i64, i64, vp, vp, vp, vp]
    lib.vts_verify_draft_workspace_bytes.restype = sz
    lib.vts_verify_draft_workspace_bytes.argtypes = [i64, i64]
    lib.vts_verify_draft.restype = ctypes.c_int
    lib.vts_verify_draft.argtypes = [vp, i32, i64, i64, vp, i64, i64, vp, vp, vp, i64, i32, i64,
                                     vp, vp, vp, vp, sz, vp]
