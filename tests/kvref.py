"""Plain float64 forms of the operators around the attention kernels, written
from their definitions (include/attn.h), for the tests."""
import math

import torch


def turn(y, cos, sin, interleaved, sign=1):
    """y [.., heads, d] float64; cos, sin [.., rot / 2] float64."""
    h = cos.shape[-1]
    i = torch.arange(h, device=y.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    c, s = cos[..., None, :], sign * sin[..., None, :]
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def norm_rope(x, w, cos, sin, norm, eps, interleaved):
    if norm:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    if w is not None:
        x = x * w
    return turn(x, cos, sin, interleaved) if cos is not None else x


def quantise(x):
    """(codes int64 [.., d], scales float64 [.., d / 32]) of a float64 tensor of
    bf16 or fp16 values."""
    g = x.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / 7).to(torch.bfloat16).double()
    bad = ~torch.isfinite(g).all(-1)
    safe = torch.where((s > 0) & ~bad, s, torch.ones_like(s))[..., None]
    c = torch.where(bad[..., None] | (s == 0)[..., None], torch.zeros_like(g), torch.round(g / safe))
    return (c.clamp(-7, 7) + 8).long().flatten(-2), torch.where(bad, torch.full_like(s, float("nan")), s)


def values(codes, scales):
    return ((codes - 8).double().unflatten(-1, (-1, 32)) * scales[..., None]).flatten(-2)


def held_at(d, is_k):
    """(byte, shift) at which dim i of a row of codes is held."""
    g = d // 32
    out = []
    for i in range(d):
        if is_k:  # word c * g + (i / 32) holds 8 dims
            nib = ((i % 32) // 8 * g + i // 32) * 8 + i % 8
        else:     # half-word r * g + (i / 32) holds 4 dims
            nib = ((i % 32) // 4 * g + i // 32) * 4 + i % 4
        out.append((nib // 2, 4 * (nib % 2)))
    byte, shift = zip(*out)
    return torch.tensor(byte), torch.tensor(shift)


def pack(codes, is_k):
    """uint8 [.., d / 2] of codes [.., d]."""
    d = codes.shape[-1]
    byte, shift = held_at(d, is_k)
    out = torch.zeros(*codes.shape[:-1], d // 2, dtype=torch.int64)
    for i in range(d):
        out[..., byte[i]] |= codes[..., i].cpu() << shift[i]
    return out.to(torch.uint8)


def unpack(rows, is_k):
    byte, shift = held_at(2 * rows.shape[-1], is_k)
    return (rows.cpu().long()[..., byte] >> shift) & 15


def plan(context, fresh, table, page, num_pages, rows, free=None, head=0):
    """Lists: (cu, seq, positions, slots, table, head)."""
    table = [list(r) for r in table]
    cu, seq, pos, slots = [0], [], [], []
    for b, (c, n) in enumerate(zip(context, fresh)):
        if free is not None:
            for blk in range(-(-c // page), -(-(c + n) // page)):
                ok = head < len(free) and 0 <= free[head] < num_pages
                table[b][blk] = free[head] if ok else -1
                head += 1
        for p in range(c, c + n):
            pg = table[b][p // page]
            pos.append(p)
            slots.append(pg * page + p % page if 0 <= pg < num_pages else -1)
        cu.append(cu[-1] + n)
        seq.append(c + n)
    pad = rows - len(pos)
    return cu, seq, (pos + [-1] * pad)[:rows], (slots + [-1] * pad)[:rows], table, head


def decode(q, kcodes, kscales, vcodes, vscales, table, lens, scale, window_left=-1, sinks=0):
    """q float64 [B, Sq, Hq, d]; codes int64 [pages, H, page, d] and scales
    float64 [pages, H, page, d / 32], all on one device.  Returns float64 o, lse,
    and for error bounds: mag = sum p |v| (like o) and big = max over visible
    keys of scale * sum |q k| (like lse)."""
    b, sq, hq, _ = q.shape
    h, page = kcodes.shape[1], kcodes.shape[2]
    grp = hq // h
    new = dict(dtype=torch.float64, device=q.device)
    o, mag = torch.zeros(b, sq, hq, vcodes.shape[3], **new), torch.zeros(b, sq, hq, vcodes.shape[3], **new)
    lse, big = torch.full((b, hq, sq), -math.inf, **new), torch.zeros(b, hq, sq, **new)
    for i in range(b):
        n = lens[i]
        if n == 0:
            continue
        at = torch.arange(n, device=q.device)
        pg = torch.tensor(table[i], device=q.device)[at // page]
        for kv in range(h):
            k = values(kcodes[pg, kv, at % page], kscales[pg, kv, at % page])
            v = values(vcodes[pg, kv, at % page], vscales[pg, kv, at % page])
            for t in range(sq):
                pos = n - sq + t
                see = at <= pos
                if window_left >= 0:
                    see &= (at >= pos - window_left) | (at < sinks)
                if not see.any():
                    continue
                hs = slice(kv * grp, (kv + 1) * grp)
                x = scale * q[i, t, hs] @ k[see].T
                e = torch.logsumexp(x, -1)
                p = torch.exp(x - e[:, None])
                lse[i, hs, t], o[i, t, hs], mag[i, t, hs] = e, p @ v[see], p @ v[see].abs()
                big[i, hs, t] = scale * (q[i, t, hs].abs() @ k[see].abs().T).amax(-1)
    return o, lse, mag, big
