"""Cases for timing the operators around a cache that is shared and bounded:
attention of a batch whose requests share a long prefix, the attention weights
that each cached token has received, and eviction of the tokens that received
least.

``own`` False: every operator in plain torch operations, in 32 bits, rounded
once at the end.  ``own`` True: the calls a user makes of this package.

The cache holds codes of 4 bits and one bf16 scale for each 32 dims of a (token,
kv head) row, value = (code - 8) * scale.  A K row of d dims is 4 * G words (G =
d / 32): word c * G + g holds dims 32 g + 8 c .. + 7, lowest nibble first.  A V
row is 8 * G half-words: half-word r * G + g holds dims 32 g + 4 r .. + 3.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_PKG = []


def _pkg():
    if not _PKG:
        from bwd_tcgen05_tmem_gb300 import kv
        _PKG.append(kv)
    return _PKG[0]


# --------------------------------------------------------------------- cases

def listed():
    return [
        # four samples of one short conversation
        dict(name="shared_samples", op="shared", dtype="bf16", groups=1, members=4, sq=1, hq=32, hkv=8, dqk=128,
             dv=128, shared=1024, own=100, ragged=False, page=64),
        # a serving batch under one system prompt, answers of very different lengths
        dict(name="shared_system_prompt", op="shared", dtype="bf16", groups=1, members=64, sq=1, hq=32, hkv=8,
             dqk=128, dv=128, shared=8192, own=2048, ragged=True, page=64),
        # a few documents, many questions about each; drafted tokens, odd lengths
        dict(name="shared_documents", op="shared", dtype="fp16", groups=5, members=13, sq=3, hq=16, hkv=4, dqk=192,
             dv=128, shared=6001, own=700, ragged=True, page=32),
        # the same with wide heads
        dict(name="shared_wide_heads", op="shared", dtype="bf16", groups=2, members=24, sq=1, hq=16, hkv=4, dqk=256,
             dv=256, shared=16384, own=256, ragged=True, page=128),
        # many requests over one long context
        dict(name="shared_long", op="shared", dtype="bf16", groups=1, members=256, sq=1, hq=32, hkv=8, dqk=128,
             dv=128, shared=32768, own=256, ragged=True, page=64),
        # weights of one step of one request
        dict(name="weights_one", op="weights", dtype="bf16", batch=1, sq=1, hq=32, hkv=8, dqk=128, ctx=1023,
             ragged=False, page=64, window=-1, sinks=0, add=True),
        # weights of one step of a batch with long contexts
        dict(name="weights_long", op="weights", dtype="bf16", batch=16, sq=1, hq=32, hkv=8, dqk=128, ctx=32768,
             ragged=False, page=64, window=-1, sinks=0, add=True),
        # the last tokens of ragged prompts give their opinion on all before them
        dict(name="weights_prompts", op="weights", dtype="fp16", batch=9, sq=32, hq=12, hkv=4, dqk=64, ctx=20001,
             ragged=True, page=32, window=-1, sinks=0, add=False),
        # one request a little over its budget
        dict(name="evict_one", op="evict", batch=1, hkv=8, dqk=128, dv=128, ctx=1087, ragged=False, page=64,
             keep=1023, first=4, recent=64),
        # a batch that runs at its budget: one page of tokens goes
        dict(name="evict_step", op="evict", batch=64, hkv=8, dqk=128, dv=128, ctx=4160, ragged=False, page=64,
             keep=4096, first=4, recent=256),
        # long prompts cut down to a budget
        dict(name="evict_prompts", op="evict", batch=16, hkv=8, dqk=128, dv=128, ctx=32768, ragged=False, page=64,
             keep=4096, first=64, recent=512),
        # ragged ones behind a shared prefix that stays, some within the budget
        dict(name="evict_odd", op="evict", batch=21, hkv=3, dqk=192, dv=128, ctx=17001, ragged=True, page=16,
             keep=2001, first=515, recent=33),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("shared", "shared", "shared", "weights", "weights", "evict", "evict"))
    dt = rng.choice(("bf16", "bf16", "fp16"))
    dqk, dv = rng.choice(((64, 64), (128, 128), (128, 128), (192, 128), (256, 256)))
    hkv = rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    group = rng.choice((1, 2, 4, 4, 5, 8, 12))
    sq = rng.choice((1, 1, 1, 2, 3, 5))
    if op == "shared":
        groups = rng.choice((1, 1, 1, 2, 3, 7))
        members = _log(rng, 1, max(2, 256 // groups))
        rows = groups * members * sq * group * hkv
        most = 256 * 32 * 32768 * 256 // (rows * (dqk + dv))  # products of the largest listed case
        shared = _log(rng, 1, max(2, min(65536 // groups, most)))
        own_ = _log(rng, sq, max(sq + 1, min(2048, 256 * 256 * 8 * 256 // (
            groups * members * hkv * (dqk + dv) * max(1, sq * group // 8)))))
        return dict(op=op, dtype=dt, groups=groups, members=members, sq=sq, hq=hkv * group, hkv=hkv, dqk=dqk, dv=dv,
                    shared=shared, own=own_, ragged=rng.random() < 0.6, page=page)
    if op == "weights":
        batch = _log(rng, 1, 64)
        sq = rng.choice((1, 1, 1, 2, 5, 16, 32))
        heavy = max(1, sq * group // 8)  # rows of queries that a token is multiplied with
        ctx = _log(rng, sq, max(sq + 1, min(65536, 16 * 32768 * 1024 // (batch * hkv * dqk * heavy))))
        window = rng.choice((-1, -1, max(1, ctx // 3)))
        return dict(op=op, dtype=dt, batch=batch, sq=sq, hq=hkv * group, hkv=hkv, dqk=dqk, ctx=ctx,
                    ragged=rng.random() < 0.6, page=page, window=window,
                    sinks=rng.choice((0, 4, 33)) if window >= 0 else 0, add=rng.random() < 0.7)
    batch = _log(rng, 1, 64)
    ctx = _log(rng, 1, max(2, min(65536, 16 * 32768 * 2048 // (batch * hkv * (dqk + dv)))))
    keep = max(1, min(ctx, 64 * 4096 * 2048 // (batch * hkv * (dqk + dv)), int(ctx * rng.uniform(0.05, 1.05))))
    return dict(op=op, batch=batch, hkv=hkv, dqk=dqk, dv=dv, ctx=ctx, ragged=rng.random() < 0.6, page=page, keep=keep,
                first=rng.choice((0, 4, keep // 5)), recent=rng.choice((0, 1, keep // 4)))


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _lens(n, most, least, ragged, g):
    """n lengths up to ``most`` (the first is that), on the host."""
    if not ragged:
        return [most] * n
    lo = max(1, least, most // 64)
    u = torch.rand(n, generator=g, device="cuda").tolist()
    out = [max(lo, int(round(lo * (most / lo) ** x))) for x in u]
    out[0] = max(most, lo)
    return out


def _side(g, pages, h, page, d, is_k, dt):
    """Quantised normal values, some pages at a time."""
    codes = torch.empty(pages, h, page, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, h, page, d // 32, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // (h * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        code, s = _quantise(torch.randn(n, h, page, d, generator=g, device="cuda").to(dt))
        codes[i:i + n], scales[i:i + n] = _pack(code, is_k), s
    return codes, scales


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"shared": _make_shared, "weights": _make_weights, "evict": _make_evict}[case["op"]](case, _gen(seed))


def _make_shared(c, g):
    """Each group's whole pages of its prefix are held once; what its last page holds of the prefix is copied for
    every request, as whoever appends to it has to do."""
    dt, h, page, m = _DT[c["dtype"]], c["hkv"], c["page"], c["members"]
    b = c["groups"] * m
    # prefixes of different lengths, members in a row
    pre = [max(1, c["shared"] * (c["groups"] - i) // c["groups"]) // page * page for i in range(c["groups"])]
    rest = [max(1, c["shared"] * (c["groups"] - i) // c["groups"]) - p for i, p in enumerate(pre)]
    own_ = _lens(b, max(c["own"], c["sq"]), c["sq"], c["ragged"], g)
    lens = [pre[i // m] + rest[i // m] + own_[i] for i in range(b)]
    cols = max(-(-n // page) for n in lens)
    need = sum(p // page for p in pre) + sum(-(-(n - pre[i // m]) // page) for i, n in enumerate(lens))
    perm = torch.randperm(need + 3, generator=g, device="cuda").tolist()
    table, at = [], 0
    heads = []
    for p in pre:
        heads.append(perm[at:at + p // page])
        at += p // page
    for i, n in enumerate(lens):
        k = -(-(n - pre[i // m]) // page)
        row = heads[i // m] + perm[at:at + k]
        at += k
        table.append(row + [0] * (cols - len(row)))
    kc, ks = _side(g, need + 3, h, page, c["dqk"], True, dt)
    vc, vs = _side(g, need + 3, h, page, c["dv"], False, dt)
    return dict(case=c, q=_normal(g, b, c["sq"], c["hq"], c["dqk"], dtype=dt, scale=1.5), table=_i32(table),
                lens=_i32(lens), starts=_i32([i * m for i in range(c["groups"] + 1)]), shared=_i32(pre),
                kc=kc, ks=ks, vc=vc, vs=vs, host=(lens, pre))


def _pages_for(lens, page, g):
    blocks = max(1, -(-max(lens) // page))
    pages = len(lens) * blocks + 3
    return torch.randperm(pages, generator=g, device="cuda")[:len(lens) * blocks].to(torch.int32).view(
        len(lens), blocks).contiguous(), pages


def _make_weights(c, g):
    dt, h, page = _DT[c["dtype"]], c["hkv"], c["page"]
    lens = _lens(c["batch"], max(c["ctx"], c["sq"]), c["sq"], c["ragged"], g)
    table, pages = _pages_for(lens, page, g)
    kc, ks = _side(g, pages, h, page, c["dqk"], True, dt)
    # V is the cache's other half; a narrow one, as nothing here reads it
    dv = 128 if c["dqk"] == 192 else c["dqk"]
    vc = torch.zeros(pages, h, page, dv // 2, dtype=torch.uint8, device="cuda")
    vs = torch.zeros(pages, h, page, dv // 32, dtype=torch.bfloat16, device="cuda")
    st = dict(case=c, q=_normal(g, c["batch"], c["sq"], c["hq"], c["dqk"], dtype=dt, scale=1.5), table=table,
              lens=_i32(lens), kc=kc, ks=ks, vc=vc, vs=vs,
              w=torch.rand(c["batch"], h, table.shape[1] * page, generator=g, device="cuda"))
    # the attention call before this one has left its log-sum-exp
    lse = torch.empty(c["batch"], c["hq"], c["sq"], device="cuda")
    for i in range(c["batch"]):
        x = torch.logsumexp(_scores(st, i), -1)
        lse[i] = x.transpose(1, 2).reshape(c["hq"], c["sq"])
    st["lse"] = lse
    return st


def _make_evict(c, g):
    h, page = c["hkv"], c["page"]
    lens = _lens(c["batch"], c["ctx"], 1, c["ragged"], g)
    table, pages = _pages_for(lens, page, g)
    cap = table.shape[1] * page
    kc, ks = _side(g, pages, h, page, c["dqk"], True, torch.bfloat16)
    vc, vs = _side(g, pages, h, page, c["dv"], False, torch.bfloat16)
    # sums of probabilities: most of them small, a few large, the longer a token is there the larger
    w = torch.exp(2 * torch.randn(c["batch"], h, cap, generator=g, device="cuda"))
    w *= torch.linspace(1, 0.05, cap, device="cuda") / cap
    spent = c["batch"] * table.shape[1] + 5
    return dict(case=c, table=table, lens=_i32(lens), w=w, w_out=torch.zeros_like(w), kc=kc, ks=ks, vc=vc, vs=vs,
                kept=torch.full((c["batch"], h, c["keep"]), -1, dtype=torch.int32, device="cuda"),
                first=torch.full((c["batch"],), c["first"], dtype=torch.int32, device="cuda"),
                free=torch.full((spent + 4,), -1, dtype=torch.int32, device="cuda"), head=_i32([spent]))


# ------------------------------------------------------------ the plain forms

def _quantise(x):
    """Codes 1..15 [.., d] and bf16 scales [.., d / 32]."""
    x = x.float().unflatten(-1, (-1, 32))
    s = (x.abs().amax(-1) / 7).to(torch.bfloat16)
    sf = s.float()[..., None]
    c = torch.where(sf > 0, torch.round(x / sf).clamp(-7, 7), torch.zeros_like(x))
    return (c + 8).to(torch.uint8).flatten(-2), s


def _pack(code, is_k):
    """Codes of a row in the cache's order, two to a byte."""
    n = code.shape[-1] // 32
    c = code.unflatten(-1, (n, 4, 8) if is_k else (n, 8, 4)).transpose(-3, -2).reshape(*code.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4)


def _unpack(b, is_k):
    """The codes of packed rows, in the order of the dims."""
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    n = c.shape[-1] // 32
    return c.unflatten(-1, (4, n, 8) if is_k else (8, n, 4)).transpose(-3, -2).flatten(-3)


def _values(codes, scales, is_k):
    c = _unpack(codes, is_k).float() - 8
    return (c.unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _rows_of(s, name, pages):
    """Rows [heads, tokens, d] that a row of pages holds."""
    v = _values(s[name + "c"][pages], s[name + "s"][pages], name == "k")
    return v.transpose(0, 1).flatten(1, 2)


def _heads(q, h):
    """[.., sq, hq, d] -> [h, .. * sq * group, d] in 32 bits."""
    n = q.shape[-2] // h
    return q.float().unflatten(-2, (h, n)).flatten(0, -4).transpose(0, 1).flatten(1, 2)


def _plain_shared(s):
    c = s["case"]
    h, page, m, sq = c["hkv"], c["page"], c["members"], c["sq"]
    grp = c["hq"] // h
    lens, pre = s["host"]
    o = torch.empty(len(lens), sq, c["hq"], c["dv"], device="cuda")
    lse = torch.empty(len(lens), c["hq"], sq, device="cuda")
    root = 1.0 / math.sqrt(c["dqk"])
    for i, p in enumerate(pre):  # a group at a time
        members = slice(i * m, (i + 1) * m)
        pages = s["table"][members].long()
        q = _heads(s["q"][members], h) * root                          # [h, m sq grp, d]
        x, v = None, None
        if p:
            x, v = q @ _rows_of(s, "k", pages[0, :p // page]).transpose(1, 2), _rows_of(s, "v", pages[0, :p // page])
        # each request's own tokens, padded to the longest
        last = -(-max(lens[members]) // page)
        pages = pages[:, p // page:last]
        k1 = _values(s["kc"][pages], s["ks"][pages], True).transpose(1, 2).flatten(2, 3)   # [m, h, n, d]
        v1 = _values(s["vc"][pages], s["vs"][pages], False).transpose(1, 2).flatten(2, 3)
        x1 = q.unflatten(1, (m, sq * grp)).transpose(0, 1) @ k1.transpose(-1, -2)           # [m, h, sq grp, n]
        at = torch.arange(x1.shape[-1], device="cuda") + p
        see = at <= (s["lens"][members].long()[:, None] - sq + torch.arange(sq, device="cuda"))[..., None]
        see = see[:, None, :, None].expand(m, 1, sq, grp, -1).flatten(2, 3)
        x1 = torch.where(see, x1, -math.inf)
        top = x1.amax(-1)
        if p:
            xp = x.unflatten(1, (m, sq * grp)).transpose(0, 1)
            top = torch.maximum(top, xp.amax(-1))
        e1 = torch.exp(x1 - top[..., None])
        total, out = e1.sum(-1), e1 @ v1
        if p:
            e = torch.exp(x - top.transpose(0, 1).flatten(1)[..., None])
            total = total + e.sum(-1).unflatten(1, (m, -1)).transpose(0, 1)
            out = out + (e @ v).unflatten(1, (m, -1)).transpose(0, 1)
        out = (out / total[..., None]).unflatten(2, (sq, grp))
        o[members] = out.transpose(1, 2).flatten(2, 3)
        lse[members] = (top + torch.log(total)).unflatten(2, (sq, grp)).transpose(2, 3).flatten(1, 2)
    return o.to(s["q"].dtype), lse


def _scores(s, i):
    """Scores of request i's queries [h, sq, grp, tokens], -inf where a token is not seen."""
    c = s["case"]
    h, page, sq = c["hkv"], c["page"], c["sq"]
    n = int(s["lens"][i])
    k = _rows_of(s, "k", s["table"][i, :-(-n // page)].long())[:, :n]
    x = (_heads(s["q"][i], h) @ k.transpose(1, 2) * (1.0 / math.sqrt(c["dqk"]))).unflatten(1, (sq, -1))
    pos = n - sq + torch.arange(sq, device="cuda")[:, None]
    at = torch.arange(n, device="cuda")
    see = at <= pos
    if c["window"] >= 0:
        see &= (at >= pos - c["window"]) | (at < c["sinks"])
    return torch.where(see[None, :, None], x, -math.inf)


def _plain_weights(s):
    c = s["case"]
    for i, n in enumerate(s["lens"].tolist()):
        lse = s["lse"][i].unflatten(0, (c["hkv"], -1)).transpose(1, 2)
        w = torch.exp(_scores(s, i) - lse[..., None]).sum((1, 2))
        if c["add"]:
            old = n - c["sq"]
            s["w"][i, :, :old] += w[:, :old]
            s["w"][i, :, old:n] = w[:, old:]
        else:
            s["w"][i, :, :n] = w
    return s["w"]


def _plain_evict(s):
    c = s["case"]
    b, h, keep, page = c["batch"], c["hkv"], c["keep"], c["page"]
    lens, cap = s["lens"].long(), s["w"].shape[2]
    at = torch.arange(cap, device="cuda")
    first = s["first"].long().clamp(max=keep)[:, None]
    recent = torch.clamp(keep - first, max=c["recent"])
    n = lens[:, None]
    must = (at < first) | ((at >= n - recent) & (at < n))
    # sorted by weight (those that must stay in front, those past the end behind), equal ones in order
    rank = torch.where(must[:, None], math.inf, s["w"])
    rank = torch.where((at < n)[:, None], rank, -1.0)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :min(keep, cap)]
    kept = order.sort(-1).values
    if kept.shape[2] < keep:
        kept = torch.cat((kept, kept.new_zeros(b, h, keep - kept.shape[2])), -1)
    new = lens.clamp(max=keep)
    i = torch.arange(keep, device="cuda")
    kept = torch.where((lens <= keep)[:, None, None], i.expand_as(kept), kept)
    live = (i < new[:, None])[:, None].expand(b, h, keep)
    bi, hi, di = torch.nonzero(live, as_tuple=True)
    si = kept[bi, hi, di]
    table = s["table"].long()
    src, dst = table[bi, si // page], table[bi, di // page]
    for name in ("kc", "ks", "vc", "vs"):
        s[name][dst, hi, di % page] = s[name][src, hi, si % page]
    s["w_out"][bi, hi, di] = s["w"][bi, hi, si]
    s["kept"].copy_(torch.where(live, kept, -1))
    # pages given back
    p0, p1 = -(-new // page), -(-lens // page)
    col = torch.arange(table.shape[1], device="cuda")
    gone = s["table"][(col >= p0[:, None]) & (col < p1[:, None])]
    head = s["head"] - gone.numel()
    s["free"][s["head"].long() - gone.numel() + torch.arange(gone.numel(), device="cuda")] = gone
    return new.int(), s["w_out"], s["kept"], s["kc"], s["ks"], s["vc"], s["vs"], s["free"], head


# ------------------------------------------------------------------ the calls

def _cache(s):
    return _pkg().KV4Cache(s["kc"], s["ks"], s["vc"], s["vs"])


def _own_shared(s):
    return _pkg().kv4_decode_shared(s["q"], _cache(s), s["table"], s["lens"], s["starts"], s["shared"])


def _own_weights(s):
    c = s["case"]
    return _pkg().kv4_weights(s["q"], _cache(s), s["table"], s["lens"], s["lse"], s["w"], window_left=c["window"],
                              sinks=c["sinks"], accumulate=c["add"])


def _own_evict(s):
    c = s["case"]
    r = _pkg().kv4_evict(_cache(s), s["table"], s["lens"], s["w"], keep=c["keep"], first=s["first"],
                         recent=c["recent"], weights_out=s["w_out"], kept=s["kept"], free_pages=s["free"],
                         free_head=s["head"])
    return r.seq_lens, r.weights, r.kept, s["kc"], s["ks"], s["vc"], s["vs"], s["free"], r.free_head


def run(state):
    op = state["case"]["op"]
    if own:
        return {"shared": _own_shared, "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"shared": _plain_shared, "weights": _plain_weights, "evict": _plain_evict}[op](state)


# --------------------------------------------------------- what a pass cannot do without

def _mean(most, ragged, least=1):
    """The mean of _lens (spread over the logarithm)."""
    lo = max(1, least, most // 64)
    return (most - lo) / math.log(most / lo) if ragged and most > lo else max(most, lo)


def work(case):
    c = case
    if c["op"] == "shared":
        row = (c["dqk"] + c["dv"]) * (0.5 + 2 / 32)
        b = c["groups"] * c["members"]
        pre = sum(max(1, c["shared"] * (c["groups"] - i) // c["groups"]) for i in range(c["groups"]))
        own_ = b * _mean(max(c["own"], c["sq"]), c["ragged"], c["sq"])
        qo = b * c["sq"] * c["hq"] * (2 * (c["dqk"] + c["dv"]) + 4)
        return {"bytes": int((pre + own_) * c["hkv"] * row + qo),
                "flops": int(2 * (pre * c["members"] + own_) * c["sq"] * c["hq"] * (c["dqk"] + c["dv"]))}
    if c["op"] == "weights":
        mean = _mean(max(c["ctx"], c["sq"]), c["ragged"], c["sq"])
        seen = min(mean, c["window"] + c["sinks"] + c["sq"]) if c["window"] >= 0 else mean
        held = seen * c["dqk"] * (0.5 + 2 / 32)
        if c["add"]:  # what no query sees stays as it is
            held += 8 * seen
        else:
            held += 4 * mean
        return {"bytes": int(c["batch"] * (c["hkv"] * held + c["sq"] * c["hq"] * (2 * c["dqk"] + 4))),
                "flops": int(2 * c["batch"] * seen * c["sq"] * c["hq"] * c["dqk"])}
    mean = _mean(c["ctx"], c["ragged"])
    over = mean > c["keep"]
    # kept rows move, but for those in front of the first that goes (the first tokens, and 1 / gone of the rest)
    moved = max(0, c["keep"] - c["first"]) if over else 0
    row = (c["dqk"] + c["dv"]) * (0.5 + 2 / 32)
    tokens = c["batch"] * c["hkv"]
    return {"bytes": int(tokens * ((4 * mean if over else 0) + 2 * row * moved + 8 * min(mean, c["keep"]))),
            "flops": 0}


# ------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_shared, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


def _reader(s, name, head):
    """f(slots) -> the rows of one kv head in 64 bits, dim by dim from where the layout puts it."""
    codes, scales = s[name + "c"], s[name + "s"]
    d = 2 * codes.shape[3]
    i = torch.arange(d, device="cuda")
    wide = 8 if name == "k" else 4  # neighbours that lie together
    at = (i % 32 // wide * (d // 32) + i // 32) * wide + i % wide

    def rows(page, offset):
        b = codes[page, head, offset].int()[:, at // 2]
        b = torch.where(at % 2 == 1, b // 16, b % 16).double() - 8
        return b * scales[page, head, offset].double().repeat_interleave(32, 1)
    return rows


def _exact_shared(s):
    c = s["case"]
    h, page, sq, m = c["hkv"], c["page"], c["sq"], c["members"]
    grp = c["hq"] // h
    lens, pre = s["host"]
    o = torch.zeros(len(lens), sq, c["hq"], c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(len(lens), c["hq"], sq, dtype=torch.float64, device="cuda")
    for head in range(h):
        rk, rv = _reader(s, "k", head), _reader(s, "v", head)
        mine = slice(head * grp, (head + 1) * grp)
        for i, n in enumerate(lens):
            p = pre[i // m]
            j = torch.arange(n, device="cuda")
            pg = s["table"][i].long()[j // page]
            if i % m == 0:  # the prefix, which the others' tables name as well
                kp, vp = rk(pg[:p], j[:p] % page), rv(pg[:p], j[:p] % page)
                first = pg[:p]
            assert torch.equal(pg[:p], first)
            k1, v1 = rk(pg[p:], j[p:] % page), rv(pg[p:], j[p:] % page)
            for t in range(sq):
                own_ = n - p - sq + t + 1
                q = s["q"][i, t, mine].double() / math.sqrt(c["dqk"])
                x = torch.cat((q @ kp.T, q @ k1[:own_].T), 1)
                e = torch.logsumexp(x, 1)
                w = torch.exp(x - e[:, None])
                lse[i, mine, t] = e
                o[i, t, mine] = w[:, :p] @ vp + w[:, p:] @ v1[:own_]
    return o, lse


def _exact_weights(s):
    c = s["case"]
    h, page, sq = c["hkv"], c["page"], c["sq"]
    grp = c["hq"] // h
    out = s["w"].double()
    for i, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n, device="cuda")
        pg = s["table"][i].long()[j // page]
        for head in range(h):
            k = _reader(s, "k", head)(pg, j % page)
            w = torch.zeros(n, dtype=torch.float64, device="cuda")
            for t in range(sq):
                here = n - sq + t
                see = j <= here
                if c["window"] >= 0:
                    see &= (here - j <= c["window"]) | (j < c["sinks"])
                for a in range(head * grp, (head + 1) * grp):
                    x = k @ s["q"][i, t, a].double() / math.sqrt(c["dqk"])
                    w += torch.where(see, torch.exp(x - s["lse"][i, a, t].double()), 0.0)
            if c["add"]:
                w[:n - sq] += out[i, head, :n - sq]
            out[i, head, :n] = w
    return out


def _exact_evict(s):
    c = s["case"]
    h, page, keep = c["hkv"], c["page"], c["keep"]
    lens, table, head = s["lens"].tolist(), s["table"].long(), int(s["head"])
    gone = []
    for i, n in enumerate(lens):
        s["kept"][i] = -1
        if n <= keep:
            s["kept"][i, :, :n] = torch.arange(n, device="cuda")
            s["w_out"][i, :, :n] = s["w"][i, :, :n]
            continue
        f = min(c["first"], keep)
        r = min(c["recent"], keep - f)
        for a in range(h):
            w = s["w"][i, a, f:n - r].double()
            # as many as there is room for: above the border all, on it the first ones
            room = keep - f - r
            stay = torch.zeros(n, dtype=torch.bool, device="cuda")
            stay[:f] = True
            stay[n - r:] = True
            if room:
                border = torch.kthvalue(w, w.numel() - room + 1).values
                on = torch.nonzero(w == border)[:, 0]
                stay[f:n - r] = w > border
                stay[f + on[:room - int((w > border).sum())]] = True
            at = torch.nonzero(stay)[:, 0]
            to = torch.arange(keep, device="cuda")
            s["kept"][i, a] = at.int()
            s["w_out"][i, a, :keep] = s["w"][i, a, at]
            for name in ("kc", "ks", "vc", "vs"):
                x = s[name][table[i, at // page], a, at % page].clone()
                s[name][table[i, to // page], a, to % page] = x
        gone += s["table"][i, -(-keep // page):-(-n // page)].tolist()
    if gone:
        s["free"][head - len(gone):head] = _i32(gone)
    return (s["lens"].clamp(max=keep), s["w_out"], s["kept"], s["kc"], s["ks"], s["vc"], s["vs"], s["free"],
            s["head"] - len(gone))
