"""A paged cache of keys and values in 4 bits, and attention over it (ctypes
binding of the attn_kv* entry points of include/attn.h).

A step of a serving loop:

  p = kv.plan(context, fresh, table, page_size=64, num_pages=n, rows=r,
              free_pages=free, free_head=head)       # pages, slots, positions
  q, k = attn.qk_norm_rope(q, k, cos, sin, positions=p.positions, ...)
  kv.kv4_write(cache, k, v, p.slots)
  o, lse = kv.kv4_decode(q, cache, table, p.seq_lens)

Longer chunks of a prompt read their prefix back instead (plan with
free_pages=None maps tokens that are held already, kv4_read returns their rows)
and use attn.fwd.  Nothing here copies to the host or synchronises, so a step
can be captured into a CUDA graph; ``status`` words are described in the header.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple, Optional

import torch

from .attn import (_CODES, _DECODE_PACK, _PLAN_PACK, Kv4CacheDesc, _sized, check_buffers, fast,
                   launch, new, on_device)

_STRIDES_PACK = struct.Struct("@2q").pack
_I32 = torch.int32


class Plan(NamedTuple):
    cu_seqlens: torch.Tensor   # int32 [batch + 1], prefix sums of the new tokens
    seq_lens: torch.Tensor     # int32 [batch], tokens held once they are written
    positions: torch.Tensor    # int32 [rows], -1 past the last token
    slots: torch.Tensor        # int32 [rows], -1 past the last token
    free_head: Optional[torch.Tensor]  # int32 [1], the next free page


def _ints(name, t, n):
    if t.dtype != _I32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{n}], not {t.dtype} {tuple(t.shape)}")


def _table(t, batch):
    """(columns, stride) of a block table."""
    if t.dim() != 2 or t.shape[0] != batch or t.dtype != _I32:
        raise ValueError("block_table must be int32 [batch, cols]")
    cols = t.shape[1]
    row, col = t.stride()
    if cols > 1 and col != 1:
        raise ValueError("rows of block_table must be contiguous")
    return cols, row


def plan(context, fresh, block_table, *, page_size, num_pages, rows, free_pages=None,
         free_head=None, out=None, status=None, stream=None):
    """Where the new tokens of a step go (attn_kv_plan).

    context, fresh: int32 [batch], tokens that each request holds and gets;
    block_table: int32 [batch, cols], updated in place; rows: room for new
    tokens; free_pages [n] and free_head [1]: the pages to take from (empty: none is
    left; None: the table is complete and only read).  ``out``: a Plan to write into."""
    check_buffers(status)
    lib = fast()
    b = context.shape[0]
    _ints("context", context, b)
    _ints("fresh", fresh, b)
    cols, row = _table(block_table, b)
    dev = on_device(context, fresh, block_table, free_pages, free_head, status)
    take = free_pages is not None
    n_free = 0
    if take:
        n_free = free_pages.numel()
        _ints("free_pages", free_pages, n_free)
        if free_head is None:
            raise ValueError("free_pages needs free_head")
        _ints("free_head", free_head, 1)
    if out is None:  # one allocation
        parts = new((2 * b + 1 + 2 * rows + take,), _I32, dev, stream).split_with_sizes(
            (b + 1, b, rows, rows, 1) if take else (b + 1, b, rows, rows))
        out = Plan(*parts) if take else Plan(*parts, None)
    else:
        on_device(context, *out)
        for name, t, n in zip(Plan._fields, out, (b + 1, b, rows, rows, 1)):
            if t is not None:
                _ints(name, t, n)
        if take and out.free_head is None:
            raise ValueError("free_pages needs out.free_head")
    # an empty tensor has no address, but NULL would mean a call without a free list
    pages = (free_pages.data_ptr() or free_head.data_ptr()) if take else None
    launch(dev, stream, lib.attn_kv_plan,
           _PLAN_PACK(b, cols, page_size, num_pages, rows, n_free, row), context.data_ptr(),
           fresh.data_ptr(), block_table.data_ptr(), pages,
           free_head.data_ptr() if take else None, out.cu_seqlens.data_ptr(),
           out.seq_lens.data_ptr(), out.positions.data_ptr(), out.slots.data_ptr(),
           out.free_head.data_ptr() if take else None,
           None if status is None else status.data_ptr())
    return out


class KV4Cache:
    """The four arrays of a cache (layout: attn_kv4_cache_t)."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        n, h, page, half_k = k_codes.shape
        half_v = v_codes.shape[3]
        for name, t, dt, last in (("k_codes", k_codes, torch.uint8, half_k),
                                  ("k_scales", k_scales, torch.bfloat16, half_k // 16),
                                  ("v_codes", v_codes, torch.uint8, half_v),
                                  ("v_scales", v_scales, torch.bfloat16, half_v // 16)):
            if t.shape != (n, h, page, last) or t.dtype != dt or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {dt} {(n, h, page, last)}")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.num_pages, self.page_size, self.heads_kv = n, page, h
        self.d_qk, self.d_v = 2 * half_k, 2 * half_v
        self.device_index = on_device(k_codes, k_scales, v_codes, v_scales)
        self.desc = Kv4CacheDesc(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                 v_scales.data_ptr(), n, page, h, self.d_qk, self.d_v)
        self._desc = ctypes.addressof(self.desc)

    @classmethod
    def empty(cls, num_pages, heads_kv, d_qk, d_v, *, page_size=64, device="cuda"):
        def one(last, dt):
            return torch.empty((num_pages, heads_kv, page_size, last), dtype=dt, device=device)
        return cls(one(d_qk // 2, torch.uint8), one(d_qk // 32, torch.bfloat16),
                   one(d_v // 2, torch.uint8), one(d_v // 32, torch.bfloat16))


def _rows(cache, name, t, tokens, d):
    if t.shape != (tokens, cache.heads_kv, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {(tokens, cache.heads_kv, d)}")
    s = t.stride()
    if s[2] != 1:
        raise ValueError("the head-dim axis must be contiguous")
    return _STRIDES_PACK(s[0], s[1])


def _move(fn, cache, k, v, slots, t, status, stream):
    check_buffers(status)
    dev = on_device(cache.k_codes, k, v, slots, status)
    _ints("slots", slots, t)
    dt = k.dtype
    if v.dtype != dt:
        raise ValueError("k and v differ in dtype")
    if dt not in _CODES:
        raise ValueError(f"unsupported dtype {dt}")
    launch(dev, stream, fn, cache._desc, _CODES[dt], t, k.data_ptr(),
           _rows(cache, "k", k, t, cache.d_qk), v.data_ptr(), _rows(cache, "v", v, t, cache.d_v),
           slots.data_ptr(), None if status is None else status.data_ptr())


def kv4_write(cache, k, v, slots, *, status=None, stream=None):
    """Quantises rows k [T, heads_kv, d_qk], v [T, heads_kv, d_v] into the cache
    at slots [T] (int32; negative: the token is left out)."""
    _move(fast().attn_kv_write, cache, k, v, slots, k.shape[0], status, stream)


def kv4_read(cache, slots, *, dtype=torch.bfloat16, k=None, v=None, status=None, stream=None):
    """The rows that the cache holds at slots [T], as (k, v) of ``dtype``.  Rows
    of negative slots stay as they are in ``k`` and ``v`` (undefined in new ones)."""
    t = slots.numel()
    if k is None:
        k = new((t, cache.heads_kv, cache.d_qk), dtype, cache.device_index, stream)
    if v is None:
        v = new((t, cache.heads_kv, cache.d_v), dtype, cache.device_index, stream)
    _move(fast().attn_kv_read, cache, k, v, slots, t, status, stream)
    return k, v


def kv4_decode(q, cache, block_table, seq_lens, *, scale=None, window_left=-1, sinks=0, out=None,
               lse=None, o_dtype=None, workspace=None, status=None, stream=None):
    """Attention of the last q.shape[1] tokens of each sequence over the cache
    (attn_kv_decode).  q [B, Sq, Hq, d_qk]; block_table int32 [B, cols];
    seq_lens int32 [B], the new tokens among them.  Returns (o [B, Sq, Hq, d_v],
    lse float32 [B, Hq, Sq])."""
    check_buffers(status, workspace)
    lib = fast()
    dev = on_device(cache.k_codes, q, block_table, seq_lens, out, lse, workspace, status)
    b, sq, hq, d = q.shape
    s0, s1, s2, s3 = q.stride()
    if d != cache.d_qk:
        raise ValueError(f"q has head dim {d}, the cache {cache.d_qk}")
    if s3 != 1:
        raise ValueError("the head-dim axis must be contiguous")
    _ints("seq_lens", seq_lens, b)
    cols, row = _table(block_table, b)
    if out is None:
        out = new((b, sq, hq, cache.d_v), o_dtype or q.dtype, dev, stream)
    elif out.shape != (b, sq, hq, cache.d_v) or out.dtype != (o_dtype or out.dtype):
        raise ValueError("out must be [B, Sq, Hq, d_v] of o_dtype")
    o0, o1, o2, o3 = out.stride()
    if o3 != 1:
        raise ValueError("the head-dim axis must be contiguous")
    if lse is None:
        lse = new((b, hq, sq), torch.float32, dev, stream)
    elif lse.shape != (b, hq, sq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B, Hq, Sq]")
    if q.dtype not in _CODES or out.dtype not in _CODES:
        raise ValueError(f"unsupported dtypes {q.dtype}, {out.dtype}")
    p = _DECODE_PACK(_CODES[q.dtype], _CODES[out.dtype], b, sq, hq, s0, s1, s2, o0, o1, o2, cols,
                     row, window_left, sinks, 1.0 / math.sqrt(d) if scale is None else scale)
    if workspace is None:
        workspace = new((_sized(dev, lib.attn_kv_decode_workspace_size, p, cache._desc),),
                        torch.uint8, dev, stream)
    launch(dev, stream, lib.attn_kv_decode, p, cache._desc, q.data_ptr(), block_table.data_ptr(),
           seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
           workspace.nbytes, None if status is None else status.data_ptr())
    return out, lse


def decode_workspace_size(q, cache, block_table, *, o_dtype=None):
    """Bytes of workspace kv4_decode needs for these tensors (any lengths)."""
    b, sq, hq, d = q.shape
    cols, row = _table(block_table, b)
    p = _DECODE_PACK(_CODES[q.dtype], _CODES[o_dtype or q.dtype], b, sq, hq, 0, 0, 0, 0, 0, 0, cols,
                     row, -1, 0, 1.0 / math.sqrt(d))
    return _sized(on_device(q), fast().attn_kv_decode_workspace_size, p, cache._desc)
