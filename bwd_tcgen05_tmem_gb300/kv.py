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
from typing import NamedTuple, Optional

import torch

from .attn import (Kv4CacheDesc, Kv4DecodeParams, KvPlanParams, _code, _sized, launch, load,
                   new, on_device, ptr)

_I64x2 = ctypes.c_int64 * 2


class Plan(NamedTuple):
    cu_seqlens: torch.Tensor   # int32 [batch + 1], prefix sums of the new tokens
    seq_lens: torch.Tensor     # int32 [batch], tokens held once they are written
    positions: torch.Tensor    # int32 [rows], -1 past the last token
    slots: torch.Tensor        # int32 [rows], -1 past the last token
    free_head: Optional[torch.Tensor]  # int32 [1], the next free page


def _ints(name, t, shape=None):
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")


def plan(context, fresh, block_table, *, page_size, num_pages, rows, free_pages=None,
         free_head=None, out=None, status=None, stream=None):
    """Where the new tokens of a step go (attn_kv_plan).

    context, fresh: int32 [batch], tokens that each request holds and gets;
    block_table: int32 [batch, cols], updated in place; rows: room for new
    tokens; free_pages [n] and free_head [1]: the pages to take from (None: the
    table is complete and only read).  ``out``: a Plan to write into."""
    lib = load()
    b = context.shape[0]
    _ints("context", context, (b,))
    _ints("fresh", fresh, (b,))
    if block_table.dim() != 2 or block_table.shape[0] != b or block_table.dtype != torch.int32:
        raise ValueError("block_table must be int32 [batch, cols]")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("rows of block_table must be contiguous")
    dev = on_device(context, fresh, block_table, free_pages, free_head, status)
    take = free_pages is not None
    if take:
        _ints("free_pages", free_pages, (free_pages.numel(),))
        if free_head is None:
            raise ValueError("free_pages needs free_head")
        _ints("free_head", free_head, (1,))
    if out is None:
        # one allocation, each part at a multiple of 4 ints
        sizes = (b + 1, b, rows, rows, 1)
        at, parts = 0, []
        buf = new(sum((n + 3) // 4 * 4 for n in sizes), torch.int32, dev, stream)
        for n in sizes:
            parts.append(buf[at:at + n])
            at += (n + 3) // 4 * 4
        out = Plan(*parts[:4], parts[4] if take else None)
    else:
        on_device(context, *out)
        for name, t, n in zip(Plan._fields, out, (b + 1, b, rows, rows, 1)):
            if t is not None:
                _ints(name, t, (n,))
        if take and out.free_head is None:
            raise ValueError("free_pages needs out.free_head")
    p = KvPlanParams(b, block_table.shape[1], page_size, num_pages, rows,
                     free_pages.numel() if take else 0, block_table.stride(0))
    launch(dev, stream, lib.attn_kv_plan, p, ptr(context), ptr(fresh), ptr(block_table),
           ptr(free_pages), ptr(free_head) if take else None, ptr(out.cu_seqlens), ptr(out.seq_lens),
           ptr(out.positions), ptr(out.slots), ptr(out.free_head) if take else None, ptr(status))
    return out


class KV4Cache:
    """The four arrays of a cache (layout: attn_kv4_cache_t)."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        on_device(k_codes, k_scales, v_codes, v_scales)
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
        self.desc = Kv4CacheDesc(ptr(k_codes), ptr(k_scales), ptr(v_codes), ptr(v_scales), n, page,
                                 h, self.d_qk, self.d_v)

    @classmethod
    def empty(cls, num_pages, heads_kv, d_qk, d_v, *, page_size=64, device="cuda"):
        def one(last, dt):
            return torch.empty((num_pages, heads_kv, page_size, last), dtype=dt, device=device)
        return cls(one(d_qk // 2, torch.uint8), one(d_qk // 32, torch.bfloat16),
                   one(d_v // 2, torch.uint8), one(d_v // 32, torch.bfloat16))


def _kv_rows(cache, name, t, tokens, d):
    if t.shape != (tokens, cache.heads_kv, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {(tokens, cache.heads_kv, d)}")
    if t.stride(2) != 1:
        raise ValueError("the head-dim axis must be contiguous")
    return _I64x2(t.stride(0), t.stride(1))


def kv4_write(cache, k, v, slots, *, status=None, stream=None):
    """Quantises rows k [T, heads_kv, d_qk], v [T, heads_kv, d_v] into the cache
    at slots [T] (int32; negative: the token is left out)."""
    lib = load()
    t = k.shape[0]
    dev = on_device(cache.k_codes, k, v, slots, status)
    _ints("slots", slots, (t,))
    if v.dtype != k.dtype:
        raise ValueError("k and v differ in dtype")
    launch(dev, stream, lib.attn_kv_write, cache.desc, _code(k.dtype), t, ptr(k),
           _kv_rows(cache, "k", k, t, cache.d_qk), ptr(v), _kv_rows(cache, "v", v, t, cache.d_v),
           ptr(slots), ptr(status))


def kv4_read(cache, slots, *, dtype=torch.bfloat16, k=None, v=None, status=None, stream=None):
    """The rows that the cache holds at slots [T], as (k, v) of ``dtype``.  Rows
    of negative slots stay as they are in ``k`` and ``v`` (undefined in new ones)."""
    lib = load()
    t = slots.numel()
    dev = on_device(cache.k_codes, slots, k, v, status)
    _ints("slots", slots, (t,))
    if k is None:
        k = new((t, cache.heads_kv, cache.d_qk), dtype, dev, stream)
    if v is None:
        v = new((t, cache.heads_kv, cache.d_v), dtype, dev, stream)
    if k.dtype != v.dtype:
        raise ValueError("k and v differ in dtype")
    launch(dev, stream, lib.attn_kv_read, cache.desc, _code(k.dtype), t, ptr(k),
           _kv_rows(cache, "k", k, t, cache.d_qk), ptr(v), _kv_rows(cache, "v", v, t, cache.d_v),
           ptr(slots), ptr(status))
    return k, v


def kv4_decode(q, cache, block_table, seq_lens, *, scale=None, window_left=-1, sinks=0, out=None,
               lse=None, o_dtype=None, workspace=None, status=None, stream=None):
    """Attention of the last q.shape[1] tokens of each sequence over the cache
    (attn_kv_decode).  q [B, Sq, Hq, d_qk]; block_table int32 [B, cols];
    seq_lens int32 [B], the new tokens among them.  Returns (o [B, Sq, Hq, d_v],
    lse float32 [B, Hq, Sq])."""
    lib = load()
    dev = on_device(cache.k_codes, q, block_table, seq_lens, out, lse, workspace, status)
    b, sq, hq, d = q.shape
    if d != cache.d_qk:
        raise ValueError(f"q has head dim {d}, the cache {cache.d_qk}")
    if q.stride(3) != 1:
        raise ValueError("the head-dim axis must be contiguous")
    _ints("seq_lens", seq_lens, (b,))
    if block_table.dim() != 2 or block_table.shape[0] != b or block_table.dtype != torch.int32:
        raise ValueError("block_table must be int32 [batch, cols]")
    cols = block_table.shape[1]
    if cols > 1 and block_table.stride(1) != 1:
        raise ValueError("rows of block_table must be contiguous")
    if out is None:
        out = new((b, sq, hq, cache.d_v), o_dtype or q.dtype, dev, stream)
    elif out.shape != (b, sq, hq, cache.d_v) or out.stride(3) != 1 or out.dtype != (o_dtype or out.dtype):
        raise ValueError("out must be [B, Sq, Hq, d_v] of o_dtype with a contiguous last axis")
    if lse is None:
        lse = new((b, hq, sq), torch.float32, dev, stream)
    elif lse.shape != (b, hq, sq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B, Hq, Sq]")
    p = Kv4DecodeParams(_code(q.dtype), _code(out.dtype), b, sq, hq, q.stride()[:3],
                        out.stride()[:3], cols, block_table.stride(0), window_left, sinks,
                        scale if scale is not None else 1.0 / math.sqrt(d))
    if workspace is None:
        workspace = new(_sized(dev, lib.attn_kv_decode_workspace_size, p, cache.desc), torch.uint8,
                        dev, stream)
    launch(dev, stream, lib.attn_kv_decode, p, cache.desc, ptr(q), ptr(block_table), ptr(seq_lens),
           ptr(out), ptr(lse), ptr(workspace), workspace.numel() * workspace.element_size(),
           ptr(status))
    return out, lse


def decode_workspace_size(q, cache, block_table, *, o_dtype=None):
    """Bytes of workspace kv4_decode needs for these tensors (any lengths)."""
    b, sq, hq, d = q.shape
    p = Kv4DecodeParams(_code(q.dtype), _code(o_dtype or q.dtype), b, sq, hq, (0, 0, 0), (0, 0, 0),
                        block_table.shape[1], block_table.stride(0), -1, 0, 1.0 / math.sqrt(d))
    return _sized(on_device(q), load().attn_kv_decode_workspace_size, p, cache.desc)
