"""Plain float64 forms of the operators on a cache that is shared and bounded (the
weights that tokens receive, eviction), written from their definitions
(include/attn.h), for the tests."""
import math

import torch

import kvref


def weights(q, kcodes, kscales, table, lens, lse, scale, window_left=-1, sinks=0):
    """q float64 [B, Sq, Hq, d]; codes and scales as in kvref.decode.  Returns lists
    (one [H, tokens] for each sequence): the weights of all of its tokens, the largest
    scale * sum |q k| of a query that sees the token, the largest |lse| of those."""
    b, sq, hq, _ = q.shape
    h, page = kcodes.shape[1], kcodes.shape[2]
    grp = hq // h
    out = []
    for i in range(b):
        n = lens[i]
        at = torch.arange(n, device=q.device)
        w = torch.zeros(3, h, n, dtype=torch.float64, device=q.device)
        if n:
            pg = torch.tensor(table[i], device=q.device)[at // page]
            for kv in range(h):
                k = kvref.values(kcodes[pg, kv, at % page], kscales[pg, kv, at % page])
                for t in range(sq):
                    pos = n - sq + t
                    see = at <= pos
                    if window_left >= 0:
                        see &= (at >= pos - window_left) | (at < sinks)
                    hs = slice(kv * grp, (kv + 1) * grp)
                    x, l = scale * q[i, t, hs] @ k.T, lse[i, hs, t].double()[:, None]
                    w[0, kv] += torch.where(see, torch.exp(x - l), 0.0).sum(0)
                    mag = scale * (q[i, t, hs].abs() @ k.abs().T)
                    w[1, kv] = torch.maximum(w[1, kv], torch.where(see, mag, 0.0).amax(0))
                    w[2, kv] = torch.maximum(w[2, kv], torch.where(see, l.abs(), 0.0).amax(0))
        out.append(w)
    return out


def stays(w, keep, first, recent):
    """Indices (ascending) of the tokens that stay of a list of weights longer than keep."""
    n = len(w)
    f = min(max(first, 0), keep)
    r = min(recent, keep - f)
    mid = sorted(range(f, n - r), key=lambda j: (1, 0, j) if math.isnan(w[j]) else (0, -w[j], j))
    return list(range(f)) + sorted(mid[:keep - f - r]) + list(range(n - r, n))


def evict(arrays, table, lens, w, w_out, keep, first, recent):
    """arrays: the cache's four, [pages, H, page, ..] on the CPU, changed in place, as is
    w_out.  Returns (seq_lens, kept [B, H, keep])."""
    page, h = arrays[0].shape[2], arrays[0].shape[1]
    kept = torch.full((len(lens), h, keep), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        t = torch.tensor(table[b])
        for a in range(h):
            at = list(range(n)) if n <= keep else stays(w[b, a, :n].tolist(), keep, first[b], recent)
            src, dst = torch.tensor(at, dtype=torch.long), torch.arange(len(at))
            kept[b, a, :len(at)] = src.int()
            for x in list(arrays):
                x[t[dst // page], a, dst % page] = x[t[src // page], a, src % page].clone()
            w_out[b, a, :len(at)] = w[b, a, src].clone()
    return [min(n, keep) for n in lens], kept


def pages_back(table, lens, keep, page):
    """The pages that an eviction gives back, in order."""
    return [table[b][j] for b, n in enumerate(lens) if n > keep for j in range(-(-keep // page), -(-n // page))]
