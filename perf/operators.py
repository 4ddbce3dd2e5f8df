"""Cases for timing the operators around the attention kernels: the norm and
rotation of queries and keys (and its gradient), the page plan of a cache, the
4-bit cache's write and read-back, and attention over that cache.

``own`` False: every operator in plain torch operations, in 32 bits, rounded
once at the end.  ``own`` True: the calls a user makes of this package.

The cache: codes are 4 bits, one bf16 scale for each 32 dims of a (token, kv
head) row, value = (code - 8) * scale.  A K row of d dims is 4 * G words (G =
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
        from bwd_tcgen05_tmem_gb300 import attn, kv
        _PKG.extend((attn, kv))
    return _PKG


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of eight requests deep in a long context
        dict(name="prep_step", op="prep", dir="fwd", dtype="bf16", batch=1, seq=8, hq=32, hkv=8, d=128,
             rot=128, inter=False, max_pos=131072, pad=0),
        # a 32K-token prompt, 32 query and 8 key heads
        dict(name="prep_prompt", op="prep", dir="fwd", dtype="bf16", batch=1, seq=32768, hq=32, hkv=8, d=128,
             rot=128, inter=False, max_pos=32768, pad=0),
        # the training step of the same heads, two sequences of 8K
        dict(name="prep_train", op="prep", dir="bwd", dtype="bf16", batch=2, seq=8192, hq=32, hkv=8, d=128,
             rot=128, inter=False, max_pos=8192, pad=0),
        # a padded odd batch, head dim 192 of which 64 rotate in adjacent pairs
        dict(name="prep_train_odd", op="prep", dir="bwd", dtype="fp16", batch=3, seq=1001, hq=6, hkv=2, d=192,
             rot=64, inter=True, max_pos=2048, pad=117),
        # page plan of a decode step
        dict(name="plan_step", op="plan", batch=64, ctx=32768, new=1, page=64, alloc=True),
        # page plan of a thousand chunked prompts
        dict(name="plan_prompts", op="plan", batch=1021, ctx=4096, new=500, page=32, alloc=True),
        # the keys and values of one decode step, stored and read back
        dict(name="cache_step", op="cache", dtype="bf16", tokens=64, hkv=8, dqk=128, dv=128, page=64),
        # those of a 32K-token prompt
        dict(name="cache_prompt", op="cache", dtype="bf16", tokens=32768, hkv=8, dqk=128, dv=128, page=64),
        # one request, a short answer
        dict(name="decode_one", op="decode", dtype="bf16", batch=1, sq=1, hq=32, hkv=8, dqk=128, dv=128,
             ctx=1023, ragged=False, page=64, window=-1, sinks=0),
        # a serving batch of very different lengths
        dict(name="decode_ragged", op="decode", dtype="bf16", batch=48, sq=1, hq=32, hkv=8, dqk=128, dv=128,
             ctx=32768, ragged=True, page=64, window=-1, sinks=0),
        # long contexts
        dict(name="decode_long", op="decode", dtype="bf16", batch=16, sq=1, hq=32, hkv=8, dqk=128, dv=128,
             ctx=32768, ragged=False, page=128, window=-1, sinks=0),
        # four drafted tokens at a time, a sliding window with first tokens kept
        dict(name="decode_draft_window", op="decode", dtype="fp16", batch=24, sq=4, hq=16, hkv=4, dqk=192, dv=128,
             ctx=16001, ragged=True, page=32, window=4095, sinks=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prep", "prep", "plan", "cache", "decode", "decode", "decode"))
    dt = rng.choice(("bf16", "bf16", "fp16"))
    if op == "prep":
        d = rng.choice((64, 128, 128, 192, 256, 512))
        hkv = rng.choice((1, 2, 3, 4, 8))
        group = rng.choice((1, 2, 4, 5, 8))
        batch = rng.choice((1, 1, 2, 3, 5))
        most = 32768 * 5120 * 2 // (3 * (hkv + hkv * group) * d * batch)
        seq = _log(rng, 1, max(2, min(32768, most)))
        return dict(op=op, dir=rng.choice(("fwd", "bwd")), dtype=dt, batch=batch, seq=seq, hq=hkv * group,
                    hkv=hkv, d=d, rot=rng.choice((d, d, d // 2)), inter=rng.random() < 0.3,
                    max_pos=max(2 * seq, 4096), pad=rng.choice((0, seq // 7)))
    if op == "plan":
        batch = _log(rng, 1, 2048)
        return dict(op=op, batch=batch, ctx=_log(rng, 1, 16384), new=_log(rng, 1, max(2, min(4096, 500000 // batch))),
                    page=rng.choice((16, 32, 64, 128, 256)), alloc=rng.random() < 0.7)
    dqk, dv = rng.choice(((64, 64), (128, 128), (128, 128), (192, 128), (256, 256)))
    hkv = rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "cache":
        return dict(op=op, dtype=dt, tokens=_log(rng, 1, 32768 * 2048 // (hkv * (dqk + dv))), hkv=hkv, dqk=dqk,
                    dv=dv, page=page)
    batch = _log(rng, 1, 64)
    sq = rng.choice((1, 1, 1, 2, 3, 5))
    group = rng.choice((1, 2, 4, 5, 8, 12))
    heavy = max(1, sq * group // 8)  # rows of queries that a token is multiplied with
    ctx = _log(rng, 1, max(2, min(65536, 16 * 32768 * 2048 // (batch * hkv * (dqk + dv) * heavy))))
    window = rng.choice((-1, -1, max(1, ctx // 3)))
    return dict(op=op, dtype=dt, batch=batch, sq=sq, hq=hkv * group, hkv=hkv, dqk=dqk, dv=dv, ctx=ctx,
                ragged=rng.random() < 0.6, page=page, window=window, sinks=rng.choice((0, 4, 33)) if window >= 0 else 0)


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _lens(case, g):
    """Tokens that each request holds, this step's among them (on the host)."""
    if not case["ragged"]:
        return [case["ctx"]] * case["batch"]
    u = torch.rand(case["batch"], generator=g, device="cuda").tolist()
    lo = max(1, case["ctx"] // 64)
    out = [int(round(lo * (case["ctx"] / lo) ** x)) for x in u]
    out[0] = case["ctx"]
    return out


def prepare(case, seed):
    g = _gen(seed)
    return {"prep": _make_prep, "plan": _make_plan, "cache": _make_cache, "decode": _make_decode}[case["op"]](case, g)


def _make_prep(c, g):
    dt, b, s, d = _DT[c["dtype"]], c["batch"], c["seq"], c["d"]
    half = c["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = torch.arange(c["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv
    # queries, keys and values come out of one projection: q and k are views of it
    qkv = _normal(g, b, s, c["hq"] + 2 * c["hkv"], d, dtype=dt)
    pos = torch.arange(s, device="cuda", dtype=torch.int32)[None] + torch.randint(
        0, max(1, c["max_pos"] - s), (b, 1), generator=g, device="cuda", dtype=torch.int32)
    pos = pos.contiguous()
    if c["pad"]:
        pos[:, s - c["pad"]:] = -1  # the rows behind each sequence
    st = dict(case=c, q=qkv[:, :, :c["hq"]], k=qkv[:, :, c["hq"]:c["hq"] + c["hkv"]], positions=pos,
              cos=ang.cos().float(), sin=ang.sin().float(),
              wq=1 + 0.2 * torch.randn(d, generator=g, device="cuda"),
              wk=1 + 0.2 * torch.randn(d, generator=g, device="cuda"),
              q_out=torch.zeros(b, s, c["hq"], d, dtype=dt, device="cuda"),
              k_out=torch.zeros(b, s, c["hkv"], d, dtype=dt, device="cuda"))
    if c["dir"] == "bwd":
        st["dq_out"] = _normal(g, b, s, c["hq"], d, dtype=dt)
        st["dk_out"] = _normal(g, b, s, c["hkv"], d, dtype=dt)
    return st


def _make_plan(c, g):
    b, page = c["batch"], c["page"]
    ctx = torch.randint(0, c["ctx"] + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    if c["new"] == 1:
        rows, new = b + 37, torch.ones(b, dtype=torch.int32, device="cuda")
    else:  # the rows are the step's capacity: what does not fit waits, the rest stays empty
        rows = c["new"] * b * 5 // 4 + 37
        new = torch.randint(0, 2 * c["new"] + 1, (b,), generator=g, device="cuda")
        new = torch.diff(new.cumsum(0).clamp(max=rows), prepend=new[:1] * 0).int()
    top = c["ctx"] + 2 * c["new"]
    blocks = -(-top // page)
    pages = b * blocks + 7
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = perm[:b * blocks].view(b, blocks).clone()
    held = -(-ctx // page)
    need = int((-(-(ctx + new) // page) - held).sum())
    free, head = None, None
    if c["alloc"]:  # pages that no request holds yet
        unused = torch.arange(blocks, device="cuda")[None] >= held[:, None]
        free = torch.cat([perm[b * blocks:], table[unused]])
        free = free[torch.randperm(free.numel(), generator=g, device="cuda")].contiguous()
        table[unused] = -1
        head = torch.randint(0, max(1, free.numel() - need), (1,), generator=g, device="cuda", dtype=torch.int32)
    return dict(case=c, ctx=ctx, new=new, table=table, free=free, head=head, pages=pages, rows=rows)


def _pages_for(lens, page, g):
    blocks = max(1, -(-max(lens) // page))
    pages = len(lens) * blocks + 3
    return torch.randperm(pages, generator=g, device="cuda")[:len(lens) * blocks].to(torch.int32).view(
        len(lens), blocks).contiguous(), pages


def _make_cache(c, g):
    dt, t, h, page = _DT[c["dtype"]], c["tokens"], c["hkv"], c["page"]
    pages = -(-t // page) + 5
    slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * page + torch.arange(page, device="cuda")
    u8, bf = dict(dtype=torch.uint8, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
    return dict(case=c, k=_normal(g, t, h, c["dqk"], dtype=dt), v=_normal(g, t, h, c["dv"], dtype=dt),
                slots=slots.view(-1)[:t].to(torch.int32).contiguous(),
                kc=torch.zeros(pages, h, page, c["dqk"] // 2, **u8), ks=torch.zeros(pages, h, page, c["dqk"] // 32, **bf),
                vc=torch.zeros(pages, h, page, c["dv"] // 2, **u8), vs=torch.zeros(pages, h, page, c["dv"] // 32, **bf))


def _make_decode(c, g):
    dt, h, page = _DT[c["dtype"]], c["hkv"], c["page"]
    lens = _lens(c, g)
    table, pages = _pages_for(lens, page, g)

    def side(d, is_k):  # quantised normal values, a few pages at a time
        codes = torch.empty(pages, h, page, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(pages, h, page, d // 32, dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 26) // (h * page * d))
        for i in range(0, pages, step):
            n = min(step, pages - i)
            code, s = _quantise(torch.randn(n, h, page, d, generator=g, device="cuda").to(dt))
            codes[i:i + n], scales[i:i + n] = _pack(code, is_k), s
        return codes, scales

    kc, ks = side(c["dqk"], True)
    vc, vs = side(c["dv"], False)
    return dict(case=c, q=_normal(g, c["batch"], c["sq"], c["hq"], c["dqk"], dtype=dt, scale=1.5), table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), kc=kc, ks=ks, vc=vc, vs=vs)


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


def _values(codes, scales, is_k, dtype=torch.float32):
    c = _unpack(codes, is_k).to(dtype) - 8
    return (c.unflatten(-1, (-1, 32)) * scales.to(dtype)[..., None]).flatten(-2)


def _turn(y, cos, sin, inter, sign):
    """The first 2 * cos.shape[-1] dims of y [.., heads, d] turned by their positions' angles."""
    r = cos.shape[-1]
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2) * sign
    a, b = (y[..., 0:2 * r:2], y[..., 1:2 * r:2]) if inter else (y[..., :r], y[..., r:2 * r])
    u, w = a * cos - b * sin, b * cos + a * sin
    t = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((t, y[..., 2 * r:]), -1)


def _prep_fwd(x, w, cos, sin, inter, eps):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    return _turn(x * r * w, cos, sin, inter, 1.0)


def _prep_bwd(x, w, dz, cos, sin, inter, eps):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    xh = x * r
    dy = _turn(dz, cos, sin, inter, -1.0)
    gh = dy * w
    return r * (gh - xh * (gh * xh).mean(-1, keepdim=True)), dy * xh


def _plain_prep(s):
    c, pos = s["case"], s["positions"].long()
    keep, at = pos >= 0, pos.clamp(min=0)
    cos, sin, here = s["cos"][at], s["sin"][at], keep[..., None, None]
    dt = s["q"].dtype
    if c["dir"] == "fwd":
        def fwd(x, w, out):
            return torch.where(here, _prep_fwd(x.float(), w, cos, sin, c["inter"], 1e-6).to(dt), out)
        return fwd(s["q"], s["wq"], s["q_out"]), fwd(s["k"], s["wk"], s["k_out"])

    def bwd(x, w, dz, out):
        dx, dw = _prep_bwd(x.float(), w, dz.float(), cos, sin, c["inter"], 1e-6)
        return torch.where(here, dx.to(dt), out), torch.where(here, dw, torch.zeros_like(dw)).sum((0, 1, 2))
    dq, dwq = bwd(s["q"], s["wq"], s["dq_out"], s["q_out"])
    dk, dwk = bwd(s["k"], s["wk"], s["dk_out"], s["k_out"])
    return dq, dk, dwq, dwk


def _plain_plan(s):
    page, ctx, new, rows = s["case"]["page"], s["ctx"].long(), s["new"].long(), s["rows"]
    seq = ctx + new
    cu = torch.cat((torch.zeros_like(seq[:1]), new.cumsum(0)))
    table = s["table"].clone()
    head = s["head"]
    if s["free"] is not None:
        held, want = -(-ctx // page), -(-seq // page)
        need = want - held
        start = need.cumsum(0) - need + s["head"]
        col = torch.arange(table.shape[1], device=table.device)[None]
        fresh = (col >= held[:, None]) & (col < want[:, None])
        at = (start[:, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)
        table = torch.where(fresh, s["free"][at], table)
        head = (s["head"] + need.sum()).to(torch.int32)
    t = torch.arange(rows, device=table.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=ctx.numel() - 1)
    pos = ctx[b] + t - cu[b]
    live = t < cu[-1]
    blk = (pos // page).clamp(max=table.shape[1] - 1)
    slots = torch.where(live, table[b, blk].long() * page + pos % page, -1)
    out = (cu.int(), seq.int(), torch.where(live, pos, -1).int(), slots.int(), table)
    return out if head is None else out + (head,)


def _plain_cache(s):
    page, slots = s["case"]["page"], s["slots"].long()
    p, o = slots // page, slots % page
    out = []
    for x, codes, scales, is_k in ((s["k"], s["kc"], s["ks"], True), (s["v"], s["vc"], s["vs"], False)):
        code, sc = _quantise(x)
        codes[p, :, o], scales[p, :, o] = _pack(code, is_k), sc
        out.append(_values(codes[p, :, o], scales[p, :, o], is_k).to(x.dtype))
    return out


def _visible(c, lens, n):
    """[batch, sq, n]: which of the cached tokens each query sees."""
    pos = lens.long()[:, None] - c["sq"] + torch.arange(c["sq"], device=lens.device)[None]
    j = torch.arange(n, device=lens.device)
    seen = j <= pos[..., None]
    if c["window"] >= 0:
        seen &= (j >= pos[..., None] - c["window"]) | (j < c["sinks"])
    return seen


def _plain_decode(s):
    c, q = s["case"], s["q"]
    b, sq, hq, d = q.shape
    h = c["hkv"]
    k = _values(s["kc"][s["table"].long()], s["ks"][s["table"].long()], True).transpose(1, 2).flatten(2, 3)
    v = _values(s["vc"][s["table"].long()], s["vs"][s["table"].long()], False).transpose(1, 2).flatten(2, 3)
    qf = q.float().view(b, sq, h, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, h, sq * (hq // h), d)
    x = (qf @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    seen = _visible(c, s["lens"], k.shape[2])[:, None, :, None].expand(b, 1, sq, hq // h, -1).flatten(2, 3)
    x = torch.where(seen, x, torch.full_like(x, float("-inf")))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    v = torch.where(seen.any(2)[..., None], v, torch.zeros_like(v))
    o = torch.where(l > 0, (p @ v) / l, torch.zeros_like(l))
    lse = (m + torch.log(l)).view(b, h, sq, hq // h).transpose(2, 3).reshape(b, hq, sq)
    return o.view(b, h, sq, hq // h, -1).permute(0, 2, 1, 3, 4).reshape(b, sq, hq, -1).to(q.dtype), lse


# ------------------------------------------------------------------ the calls

def _own_prep(s):
    attn, c = _pkg()[0], s["case"]
    if c["dir"] == "fwd":
        return attn.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], positions=s["positions"], wq=s["wq"], wk=s["wk"],
                                 eps=1e-6, interleaved=c["inter"], q_out=s["q_out"], k_out=s["k_out"])
    return attn.qk_norm_rope_bwd(s["q"], s["k"], s["cos"], s["sin"], s["dq_out"], s["dk_out"],
                                 positions=s["positions"], wq=s["wq"], wk=s["wk"], eps=1e-6, interleaved=c["inter"],
                                 dq=s["q_out"], dk=s["k_out"])


def _own_plan(s):
    kv = _pkg()[1]
    r = kv.plan(s["ctx"], s["new"], s["table"], page_size=s["case"]["page"], num_pages=s["pages"], rows=s["rows"],
                free_pages=s["free"], free_head=s["head"])
    out = (r.cu_seqlens, r.seq_lens, r.positions, r.slots, s["table"])
    return out if s["free"] is None else out + (r.free_head,)


def _own_cache(s):
    kv = _pkg()[1]
    cache = kv.KV4Cache(s["kc"], s["ks"], s["vc"], s["vs"])
    kv.kv4_write(cache, s["k"], s["v"], s["slots"])
    return kv.kv4_read(cache, s["slots"], dtype=s["k"].dtype)


def _own_decode(s):
    kv, c = _pkg()[1], s["case"]
    cache = kv.KV4Cache(s["kc"], s["ks"], s["vc"], s["vs"])
    return kv.kv4_decode(s["q"], cache, s["table"], s["lens"], window_left=c["window"], sinks=c["sinks"])


def run(state):
    op = state["case"]["op"]
    if own:
        f = {"prep": _own_prep, "plan": _own_plan, "cache": _own_cache, "decode": _own_decode}[op]
    else:
        f = {"prep": _plain_prep, "plan": _plain_plan, "cache": _plain_cache, "decode": _plain_decode}[op]
    return f(state)


# --------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "prep":
        el = c["batch"] * (c["seq"] - c["pad"]) * (c["hq"] + c["hkv"]) * c["d"]
        n = c["batch"] * c["seq"]
        table = 2 * 4 * (c["rot"] // 2) * min(n, c["max_pos"])
        if c["dir"] == "fwd":
            return {"bytes": 4 * el + 4 * n + table, "flops": 8 * el}
        return {"bytes": 6 * el + 4 * n + table, "flops": 18 * el}
    if c["op"] == "plan":
        tokens = c["batch"] * c["new"]
        return {"bytes": 8 * tokens + 4 * 4 * c["batch"] + 4 * tokens // c["page"], "flops": 0}
    if c["op"] == "cache":
        n = c["tokens"] * c["hkv"] * (c["dqk"] + c["dv"])
        held = n // 2 + 2 * (n // 32)
        return {"bytes": 2 * (2 * n + held) + 8 * c["tokens"], "flops": 4 * n}
    mean = c["ctx"]
    if c["ragged"]:  # lengths spread over the logarithm between ctx / 64 and ctx
        lo = max(1, c["ctx"] // 64)
        mean = (c["ctx"] - lo) / math.log(c["ctx"] / lo) if c["ctx"] > lo else c["ctx"]
    if c["window"] >= 0:
        mean = min(mean, c["window"] + c["sinks"] + c["sq"])
    tokens = c["batch"] * mean
    row = (c["dqk"] + c["dv"]) * (0.5 + 2 / 32)
    qo = 2 * c["batch"] * c["sq"] * c["hq"] * (c["dqk"] + c["dv"])
    return {"bytes": int(tokens * c["hkv"] * row + qo + 4 * tokens / c["page"]),
            "flops": int(2 * tokens * c["sq"] * c["hq"] * (c["dqk"] + c["dv"]))}


# ------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"prep": _exact_prep, "plan": lambda s: None, "cache": _exact_cache, "decode": _exact_decode}[case["op"]](s)


def _exact_prep(s):
    c = s["case"]
    d, r = c["d"], c["rot"] // 2
    pos = s["positions"].reshape(-1).long()
    rows = torch.nonzero(pos >= 0)[:, 0]
    cs, sn = s["cos"][pos[rows]].double(), s["sin"][pos[rows]].double()
    first = torch.arange(r, device="cuda") * (2 if c["inter"] else 1)
    second = first + (1 if c["inter"] else r)
    outs, sums = [], []
    for x, w, dz, held in ((s["q"], s["wq"], s.get("dq_out"), s["q_out"]), (s["k"], s["wk"], s.get("dk_out"), s["k_out"])):
        w = w.double()
        out, dw = held.double().flatten(0, 1), torch.zeros(d, dtype=torch.float64, device="cuda")
        for i in range(x.shape[2]):  # head by head
            xi = x[:, :, i].reshape(-1, d)[rows].double()
            norm = (xi.pow(2).sum(1, keepdim=True) / d + 1e-6).sqrt()
            n = xi / norm
            if c["dir"] == "fwd":
                y = n * w
                z = y.clone()
                z[:, first] = cs * y[:, first] - sn * y[:, second]
                z[:, second] = sn * y[:, first] + cs * y[:, second]
            else:
                t = dz[:, :, i].reshape(-1, d)[rows].double()
                dy = t.clone()
                dy[:, first] = cs * t[:, first] + sn * t[:, second]
                dy[:, second] = cs * t[:, second] - sn * t[:, first]
                dw += (dy * n).sum(0)
                e = dy * w
                z = (e - n * ((e * n).sum(1, keepdim=True) / d)) / norm
            out[rows, i] = z
        outs.append(out.view(held.shape))
        sums.append(dw)
    return tuple(outs) if c["dir"] == "fwd" else tuple(outs + sums)


def _exact_cache(s):
    out = []
    for x in (s["k"], s["v"]):
        g = x.double().view(*x.shape[:-1], -1, 32)
        step = (g.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).double()
        near = torch.where(step > 0, torch.round(g / step), 0.0).clamp(-7, 7)
        out.append((near * step).view(x.shape))
    return out


def _exact_decode(s):
    c = s["case"]
    page, h = c["page"], c["hkv"]
    grp = c["hq"] // h
    dev = "cuda"
    # where dim i of a K or a V row is held: byte and shift
    i = torch.arange(c["dqk"], device=dev)
    at_k = (i % 32 // 8 * (c["dqk"] // 32) + i // 32) * 8 + i % 8
    i = torch.arange(c["dv"], device=dev)
    at_v = (i % 32 // 4 * (c["dv"] // 32) + i // 32) * 4 + i % 4

    def rows(codes, scales, at, d, p, o, head):
        b = codes[p, head, o].long()[:, at // 2]
        b = torch.where(at % 2 == 1, b // 16, b % 16).double() - 8
        return b * scales[p, head, o].double()[:, torch.arange(d, device=dev) // 32]

    o = torch.zeros(c["batch"], c["sq"], c["hq"], c["dv"], dtype=torch.float64, device=dev)
    lse = torch.full((c["batch"], c["hq"], c["sq"]), -math.inf, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n, device=dev)
        p = s["table"][b].long()[j // page]
        for head in range(h):
            k = rows(s["kc"], s["ks"], at_k, c["dqk"], p, j % page, head)
            v = rows(s["vc"], s["vs"], at_v, c["dv"], p, j % page, head)
            for t in range(c["sq"]):
                here = n - c["sq"] + t
                if here < 0:
                    continue
                see = j <= here
                if c["window"] >= 0:
                    see &= (here - j <= c["window"]) | (j < c["sinks"])
                x = s["q"][b, t, head * grp:(head + 1) * grp].double() @ k[see].T / math.sqrt(c["dqk"])
                e = torch.logsumexp(x, 1)
                lse[b, head * grp:(head + 1) * grp, t] = e
                o[b, t, head * grp:(head + 1) * grp] = torch.exp(x - e[:, None]) @ v[see]
    return o, lse
