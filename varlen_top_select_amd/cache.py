"""Filling a paged KV cache, reading it back, and prompts (see include/vts.h).

    write_cache(q, k, v, slots, k_cache, v_cache, ...)   -> (q_out, k_out | None)
    read_cache(k_cache, v_cache, slots, ...)             -> (k, v)
    prompt_attention(q, k, v, cu_seqlens, ...)           -> (out, lse | None)
    rotary_table(max_position, rot, ...)                 -> table
    page_slots(page_table, page_size, positions)         -> slots

A cache is a pair of 4-D tensors ``[num_pages, page_size, kv_heads, head_dim]`` as
in ``varlen_top_select_amd.decode``, bfloat16 or float16, or microscaled: uint8 rows of
head_dim bytes (8 bits to an element, E4M3) or head_dim / 2 (4 bits, E2M1, the first of
two in the low half of a byte), strides that are multiples of 16, with uint8 scales
``[num_pages, page_size, kv_heads, head_dim / 32]``, a power of two (E8M0, 2^(x - 127))
to each 32 elements.  head_dim is 64 or 128.  ``torch.zeros`` makes an empty one.

A slot is ``page * page_size + position in the page``, as ``topk_page_table_transform``
writes them; -1 is no slot.  A request's way is: ``write_cache`` with its prompt's
tokens and ``prompt_attention`` over them (behind what ``read_cache`` returns of an
earlier part), then ``write_cache`` and ``tree_attention`` for each decode step.

The operators serve and have no derivatives: their outputs carry no gradient.
"""
from __future__ import annotations

import math
import struct

import torch

from . import _DTYPE, _check, library
from .decode import _CACHE, _cache, _meets, _micro, _run, _tensor

__all__ = ["write_cache", "read_cache", "prompt_attention", "rotary_table", "page_slots"]

_TOKENS = struct.Struct("@QQQqqqqqqQQdQqQQqQQiiii")  # vts_new_tokens
_PROMPTS = struct.Struct("@QQQqqqqqqQQqqqiiii")      # vts_prompts


def _slot_cache(k_cache, v_cache, k_scales, v_scales, dtype):
    """(vts_paged_cache as bytes, vts_microscales as bytes or None, device index, dtype,
    kv_heads, head_dim) of a cache without a page table"""
    if k_scales is not None or v_scales is not None:
        ks, vs, scales, index, head_dim = _micro(k_cache, v_cache, k_scales, v_scales)
        if dtype is not torch.bfloat16 and dtype is not torch.float16:
            raise ValueError("a microscaled cache is written from and read as bfloat16 or float16")
    else:
        ks, scales = _cache("k_cache", k_cache), None
        vs = _cache("v_cache", v_cache, k_cache)
        index, head_dim = k_cache.get_device(), k_cache.shape[3]
        if v_cache.shape != k_cache.shape:
            raise ValueError("v_cache must have the shape of k_cache")
        if dtype is not None and dtype is not k_cache.dtype:
            raise ValueError("a 16-bit cache is written from and read as its own dtype")
        dtype = k_cache.dtype
    pages, page_size, kv_heads = k_cache.shape[:3]
    packed = _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), *ks, *vs, 0, 0, 0, 0, pages, page_size,
                         kv_heads, head_dim, 0, _DTYPE[dtype])
    return packed, scales, index, dtype, kv_heads, head_dim


def _heads(name, t, dtype, index):
    """The shape and the strides of rows [tokens, heads, head_dim] (0 for a dimension of one)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D tensor [tokens, heads, head_dim]")
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{index}")
    n, h, d = shape = t.shape
    a, b, c = t.stride()
    if n <= 1:
        a = 0
    if h <= 1:
        b = 0
        if h < 1:
            raise ValueError(f"{name} must have heads")
    if (a | b) & 7 or c != 1 or n and t.data_ptr() & 15:
        raise ValueError(f"{name} rows must be contiguous, 16-byte aligned, with strides that are "
                         "multiples of 8 elements")
    return shape, (a, b)


def _keys(name, t, dtype, index, shape):
    """The strides of such rows of a shape."""
    got, steps = _heads(name, t, dtype, index)
    if got != shape:
        raise ValueError(f"{name} must have the shape {shape}")
    return steps


def _apart(name, out, *others):
    if any(t is not None and _meets(out, t if t.dim() == 4 else t.unsqueeze(0)) for t in others):
        raise ValueError(f"{name} must not overlap the inputs or the caches")


def _own_rows(*pairs):
    """That the rows written of each pair of caches (or scales) are apart, as far as their addresses and
    steps of 0 tell: two threads would write one of them in any order."""
    for k, v in pairs:
        if k is None:
            continue
        if k.numel() and k.data_ptr() == v.data_ptr():
            raise ValueError("k_cache and v_cache, or their scales, must not overlap where they are written")
        for t in (k, v):
            if 0 in t.stride() and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
                raise ValueError("k_cache, v_cache and their scales must not overlap themselves where they are written")


def write_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                k_cache: torch.Tensor, v_cache: torch.Tensor, *, k_scales: torch.Tensor | None = None,
                v_scales: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                rotary: torch.Tensor | None = None, interleaved: bool = False,
                q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, eps: float = 1e-6,
                q_out: torch.Tensor | None = None, return_k: bool = False, stream=None):
    """Normalises the heads of q[tokens, heads, head_dim] and k[tokens, kv_heads, head_dim]
    (``q_norm``, ``k_norm``: weights [head_dim], either or none), turns them by the angles of
    ``positions`` (int32 [tokens]) in ``rotary`` (float32 [max_position, rot], cosines then
    sines; pairs (i, i + rot / 2), or neighbours if ``interleaved``), and writes k and v to the
    ``slots`` (int32 [tokens]) of the caches (vts_write_cache in include/vts.h), whose rows must not
    overlap each other's.  A slot outside the cache is not written; the others must be distinct.  A token whose position is outside the
    table is not written and gets zeros.  Returns the queries, in ``q_out`` if given, and with
    ``return_k`` the keys as they are before they are cut to the cache's bits, else None."""
    if not isinstance(q, torch.Tensor):
        raise ValueError("q must be a 3-D tensor [tokens, heads, head_dim]")
    cache, scales, index, dtype, kv_heads, head_dim = _slot_cache(k_cache, v_cache, k_scales, v_scales, q.dtype)
    _own_rows((k_cache, v_cache), (k_scales, v_scales))
    (tokens, heads, dim), qs = _heads("q", q, dtype, index)
    if dim != head_dim:
        raise ValueError("q must have the cache's head_dim")
    ks = _keys("k", k, dtype, index, (tokens, kv_heads, head_dim))
    vs = _keys("v", v, dtype, index, (tokens, kv_heads, head_dim))
    _tensor("slots", slots, torch.int32, (tokens,), index)
    if (positions is None) != (rotary is None):
        raise ValueError("positions and rotary must be given together")
    rot = max_position = 0
    if rotary is not None:
        if not isinstance(rotary, torch.Tensor) or rotary.dim() != 2:
            raise ValueError("rotary must be a float32 tensor [max_position, rot]")
        max_position, rot = rotary.shape
        _tensor("rotary", rotary, torch.float32, (max_position, rot), index)
        if max_position < 1 or rot < 16 or rot % 16 or rot > head_dim or rotary.data_ptr() & 15:
            raise ValueError("rotary must be 16-byte aligned, not empty, with a multiple of 16 columns, "
                             "at most head_dim")
        _tensor("positions", positions, torch.int32, (tokens,), index)
    qn = kn = norm = 0
    if q_norm is not None or k_norm is not None:
        kind = (k_norm if q_norm is None else q_norm).dtype
        if kind is not dtype and kind is not torch.float32:
            raise ValueError("q_norm and k_norm must be float32 or of q's dtype, both the same")
        norm = _DTYPE[kind]
        if q_norm is not None:
            qn = _tensor("q_norm", q_norm, kind, (head_dim,), index).data_ptr()
        if k_norm is not None:
            kn = _tensor("k_norm", k_norm, kind, (head_dim,), index).data_ptr()
        if (qn | kn) & 15:
            raise ValueError("q_norm and k_norm must be 16-byte aligned")
    if not 0 <= eps < math.inf:
        raise ValueError("eps must be a finite number, not negative")
    if q_out is not None:
        _tensor("q_out", q_out, dtype, (tokens, heads, head_dim), index)
        if q_out.data_ptr() & 15:
            raise ValueError("q_out must be 16-byte aligned")
        _apart("q_out", q_out, q, k, v, k_cache, v_cache, k_scales, v_scales)
    lib = library()

    def call(sp):
        out = q.new_empty((tokens, heads, head_dim)) if q_out is None else q_out
        k_out = q.new_empty((tokens, kv_heads, head_dim)) if return_k else None
        packed = _TOKENS.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), *qs, *ks, *vs, qn, kn, eps,
            0 if rotary is None else rotary.data_ptr(), max_position,
            0 if positions is None else positions.data_ptr(), slots.data_ptr(), tokens, out.data_ptr(),
            0 if k_out is None else k_out.data_ptr(), heads, norm, rot, bool(interleaved))
        _check("vts_write_cache", lib.vts_write_cache(cache, scales, packed, sp))
        return out, k_out

    return _run(stream, index, call)


def read_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor, *,
               k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None,
               dtype: torch.dtype | None = None, stream=None):
    """The cached rows of ``slots`` (int32, any shape), zeros for a slot outside the cache
    (vts_read_cache in include/vts.h): k and v [*slots.shape, kv_heads, head_dim], of the cache's
    dtype or, of a microscaled cache, ``dtype`` (bfloat16 unless given)."""
    micro = k_scales is not None or v_scales is not None
    if dtype is None and micro:
        dtype = torch.bfloat16
    cache, scales, index, dtype, kv_heads, head_dim = _slot_cache(k_cache, v_cache, k_scales, v_scales, dtype)
    if (not isinstance(slots, torch.Tensor) or slots.dtype is not torch.int32 or slots.get_device() != index
            or not slots.is_contiguous()):
        raise ValueError(f"slots must be a contiguous int32 tensor on cuda:{index}")
    lib = library()
    shape = (*slots.shape, kv_heads, head_dim)

    def call(sp):
        k, v = k_cache.new_empty(shape, dtype=dtype), k_cache.new_empty(shape, dtype=dtype)
        _check("vts_read_cache", lib.vts_read_cache(cache, scales, slots.data_ptr(), slots.numel(),
                                                    k.data_ptr(), v.data_ptr(), sp))
        return k, v

    return _run(stream, index, call)


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                     cu_seqlens_k: torch.Tensor | None = None, causal: bool = True,
                     scale: float | None = None, out: torch.Tensor | None = None,
                     return_lse: bool = False, stream=None):
    """Attention of packed prompts (vts_prompt_attention in include/vts.h): sequence b has the rows
    cu_seqlens[b] to cu_seqlens[b + 1] of q[tokens, heads, head_dim] and those of ``cu_seqlens_k``
    (``cu_seqlens`` if None) of k and v[.., kv_heads, head_dim]; ``causal``: its queries are the last
    of its keys, and each sees the keys up to its own.  cu_seqlens are int32 [batch + 1], ascending.
    Returns the outputs, in ``out`` if given, which must not overlap the inputs, and the rows'
    log-sum-exp [tokens, heads] or None.  Rows of no sequence are left as they were in ``out``, and
    are zeros (-inf) in new outputs."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be on the GPU")
    dtype, index = q.dtype, q.get_device()
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("q dtype must be bfloat16 or float16")
    (total_q, heads, head_dim), qs = _heads("q", q, dtype, index)
    if head_dim != 64 and head_dim != 128:
        raise ValueError("head_dim must be 64 or 128")
    (total_k, kv_heads, dim), ks = _heads("k", k, dtype, index)
    if dim != head_dim:
        raise ValueError("k must have q's head_dim")
    vs = _keys("v", v, dtype, index, (total_k, kv_heads, dim))
    if heads % kv_heads:
        raise ValueError("the query heads must be a multiple of the KV heads")
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be an int32 tensor [batch + 1]")
    batch = cu_seqlens.shape[0] - 1
    _tensor("cu_seqlens", cu_seqlens, torch.int32, (batch + 1,), index)
    _tensor("cu_seqlens_k", cu_seqlens_k, torch.int32, (batch + 1,), index)
    if out is not None:
        _tensor("out", out, dtype, (total_q, heads, head_dim), index)
        if out.data_ptr() & 15:
            raise ValueError("out must be 16-byte aligned")
        _apart("out", out, q, k, v)
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    lib = library()
    need = lib.vts_prompt_attention_workspace_bytes(batch, total_q, total_k, heads, kv_heads, head_dim)
    packed = _PROMPTS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), *qs, *ks, *vs, cu_seqlens.data_ptr(),
                           cu_seqlens_k.data_ptr(), batch, total_q, total_k, heads, kv_heads, head_dim,
                           _DTYPE[dtype])

    def call(sp):
        o = q.new_empty((total_q, heads, head_dim)) if out is None else out
        lse = None
        if return_lse:  # (beside outputs that are left as they were, rows of no sequence are not written)
            lse = (q.new_empty((total_q, heads), dtype=torch.float32) if out is None
                   else q.new_full((total_q, heads), -math.inf, dtype=torch.float32))
        # (of any contents, so it is the call's own, also in a captured graph)
        ws = q.new_empty(need, dtype=torch.uint8) if need else None
        _check("vts_prompt_attention", lib.vts_prompt_attention(
            packed, bool(causal), scale, o.data_ptr(), lse.data_ptr() if return_lse else None,
            out is None, ws.data_ptr() if need else None, need, sp))
        return o, lse

    return _run(stream, index, call)


def rotary_table(max_position: int, rot: int, *, base: float = 10000.0, device=None) -> torch.Tensor:
    """float32 [max_position, rot]: cosines, then sines, of position * base^(-2 i / rot), i < rot / 2,
    as ``write_cache`` takes them.  The angles are computed in 64 bits: in 32 they are off by 2^-24 of
    their size, 0.008 at position 131072."""
    if rot < 16 or rot % 16 or max_position < 1:
        raise ValueError("rot must be a multiple of 16, and max_position at least 1")
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * base ** (-i / rot)
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()


def page_slots(page_table: torch.Tensor, page_size: int, positions: torch.Tensor) -> torch.Tensor:
    """int32 slots of ``positions`` [batch, n] in the requests' pages (page_table [batch, width]): -1
    where a position is negative or past the table, its entry is negative, or the slot no int32."""
    if page_table.dim() != 2 or positions.dim() != 2 or positions.shape[0] != page_table.shape[0]:
        raise ValueError("page_table and positions must be 2-D, with a row to each request")
    if page_size < 1:
        raise ValueError("page_size must be positive")
    if page_table.shape[1] == 0:
        return torch.full_like(positions, -1, dtype=torch.int32)
    pos = positions.long()
    page = torch.div(pos, page_size, rounding_mode="floor")
    known = (pos >= 0) & (page < page_table.shape[1])
    entry = page_table.long().gather(1, torch.where(known, page, 0))
    # (an entry whose slots all pass 32 bits may wrap in the product)
    known = known & (entry >= 0) & (entry <= (2**31 - 1) // page_size)
    slot = entry * page_size + pos % page_size
    return torch.where(known & (slot < 2**31), slot, -1).to(torch.int32)


def declare(lib):
    """Argument types of the C entry points."""
    import ctypes

    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.vts_write_cache.restype = ctypes.c_int
    lib.vts_write_cache.argtypes = [vp, vp, vp, vp]
    lib.vts_read_cache.restype = ctypes.c_int
    lib.vts_read_cache.argtypes = [vp, vp, vp, i64, vp, vp, vp]
    lib.vts_prompt_attention.restype = ctypes.c_int
    lib.vts_prompt_attention.argtypes = [vp, i32, f32, vp, vp, i32, vp, ctypes.c_size_t, vp]
    lib.vts_prompt_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.vts_prompt_attention_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i32]
