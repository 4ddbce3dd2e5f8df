"""A serving loop's use of the operators on a shared and bounded cache together: requests
over one system prompt that is held once, each cut down to a budget whenever a page over
it is full.  Every step is compared with the float64 forms on what the cache holds (bounds
as in test_gpu_kv_shared.py and test_gpu_kv_bounded.py), and the pages are counted."""
import math

import pytest
import torch

import boundedref
import kvref
from bwd_tcgen05_tmem_gb300 import attn, kv
from test_gpu_kv import BF, empty_cache, i32
from test_gpu_kv_shared import within

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, B, PAGES = 8, 2, 128, 32, 5, 48
PROMPT, OWN, KEEP, RECENT, COLS, ROWS = 96, [50, 20, 3, 54, 33], 150, 16, 8, 180


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bwd_tcgen05_tmem_gb300 import build
    build.build()
    attn.load()


class Loop:
    """The loop's state in tensors that stay where they are, so that a step of it can be captured."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.cache = empty_cache(PAGES, HK, D, D, PAGE)
        self.table = torch.full((B, COLS), -1, dtype=torch.int32, device="cuda")
        self.free, self.head = torch.randperm(PAGES, generator=g).int().cuda(), i32([0])
        self.ctx, self.first = i32([0] * B), i32([PROMPT] * B)
        self.starts, self.prompt = i32([0, B]), i32([PROMPT])
        self.w = torch.zeros(B, HK, COLS * PAGE, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cos, self.sin = attn.rope_tables(COLS * PAGE, D)
        self.g = g
        # the prompt, written by the first request; the others name its pages
        self.write(i32([PROMPT] + [0] * (B - 1)), self.inputs())
        self.table[:, :PROMPT // PAGE] = self.table[0, :PROMPT // PAGE].clone()
        self.ctx.fill_(PROMPT)
        q = self.write(i32(OWN), self.inputs())
        # the last query of each request: what it looks at starts the weights
        self.attend(q, False)

    def inputs(self):
        return torch.randn(ROWS, HQ + 2 * HK, D, generator=self.g).to(BF).cuda()

    def write(self, new, qkv):
        p = kv.plan(self.ctx, new, self.table, page_size=PAGE, num_pages=PAGES,
                    rows=ROWS, free_pages=self.free, free_head=self.head, status=self.status)
        q, k = attn.qk_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HK], self.cos, self.sin, positions=p.positions,
                                 status=self.status)
        kv.kv4_write(self.cache, k, qkv[:, HQ + HK:], p.slots, status=self.status)
        self.ctx.copy_(p.seq_lens)
        self.head.copy_(p.free_head)
        return q[(p.cu_seqlens[1:].long() - 1).clamp(min=0)][:, None]

    def attend(self, q, accumulate=True):
        o, lse = kv.kv4_decode_shared(q, self.cache, self.table, self.ctx, self.starts, self.prompt,
                                      status=self.status)
        kv.kv4_weights(q, self.cache, self.table, self.ctx, lse, self.w, accumulate=accumulate, status=self.status)
        return o, lse

    def cut(self):
        r = kv.kv4_evict(self.cache, self.table, self.ctx, self.w, keep=KEEP, first=self.first, recent=RECENT,
                         free_pages=self.free, free_head=self.head, status=self.status)
        self.ctx.copy_(r.seq_lens)
        self.head.copy_(r.free_head)
        return r.kept

    def step(self, new, qkv):
        q = self.write(new, qkv)
        o, lse = self.attend(q)
        return q, o, lse, self.cut()

    def state(self):
        c = self.cache
        return [c.k_codes, c.k_scales.view(torch.int16), c.v_codes, c.v_scales.view(torch.int16), self.table, self.free,
                self.head, self.ctx, self.w]


def arrays(cache):
    return [x.cpu().view(torch.int16) if x.dtype == BF else x.cpu().clone()
            for x in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def check_step(x, new, qkv):
    before_w = x.w.clone()
    q = x.write(new, qkv)
    lens, table, c = x.ctx.tolist(), x.table.tolist(), x.cache
    prompt = arrays(c)
    o, lse = x.attend(q)
    kc, vc = kvref.unpack(c.k_codes, True).cuda(), kvref.unpack(c.v_codes, False).cuda()
    ks, scale = c.k_scales.double(), 1 / math.sqrt(D)
    within(o, lse, kvref.decode(q.double(), kc, ks, vc, c.v_scales.double(), table, lens, scale))
    for i, (n, (ref, big, top)) in enumerate(zip(lens, boundedref.weights(q.double(), kc, ks, table, lens, lse, scale))):
        old = before_w[i, :, :n].double()
        old[:, n - 1:] = 0.0
        tol = ref * (2.0 ** -20 * big + 2.0 ** -21 * (big + top) + 2.0 ** -21 + 4 * 2.0 ** -24) + (old + ref) * 2.0 ** -23
        assert ((x.w[i, :, :n].double() - old - ref).abs() <= tol + 2.0 ** -118).all()
    # the cut moves bits
    want, w, free, head = arrays(c), x.w.cpu(), x.free.tolist(), x.head.tolist()[0]
    out = w.clone()
    seq, kept = boundedref.evict(want, table, lens, w, out, KEEP, [PROMPT] * B, RECENT)
    back = boundedref.pages_back(table, lens, KEEP, PAGE)
    got = x.cut()
    attn.query_status(x.status)
    assert torch.equal(got.cpu(), kept) and x.ctx.tolist() == seq and torch.equal(x.w.cpu(), out)
    assert all(torch.equal(a, b) for a, b in zip(arrays(c), want))
    assert x.head.tolist() == [head - len(back)] and x.free.tolist() == free[:head - len(back)] + back + free[head:]
    # the prompt's pages are as they were, every other page is held once or free
    for a, b in zip(arrays(c), prompt):
        t = torch.tensor(table[0][:PROMPT // PAGE])
        assert torch.equal(a[t], b[t])
    held = table[0][:PROMPT // PAGE]
    for row, n in zip(table, seq):
        assert row[:PROMPT // PAGE] == table[0][:PROMPT // PAGE]
        held = held + row[PROMPT // PAGE:-(-n // PAGE)]
    assert sorted(held + x.free.tolist()[x.head.tolist()[0]:]) == list(range(PAGES))
    return len(back)


def test_steps_over_a_shared_prompt_within_a_budget():
    x = Loop(seed=21)
    back = 0
    for i in range(24):
        back += check_step(x, i32([1, 1, 1, 1, 1] if i % 3 else [1, 7, 40, 1, 1]), x.inputs())
    assert back > 3  # pages came back, and were used again: every request is at its budget
    assert x.ctx.tolist() == [KEEP] * B


def test_captured_steps_are_the_same():
    """The same loop with its step in a CUDA graph, replayed: every bit of its state."""
    a, b = Loop(seed=22), Loop(seed=22)
    assert all(torch.equal(s, t) for s, t in zip(a.state(), b.state()))
    new, qkv = i32([1] * B), a.inputs()
    saved = [t.clone() for t in b.state()]
    b.step(new, qkv)  # (before the capture: what is loaded at first use)
    torch.cuda.synchronize()
    for t, s in zip(b.state(), saved):
        t.copy_(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b.step(new, qkv)
    for t, s in zip(b.state(), saved):
        t.copy_(s)
    for i in range(20):
        new.copy_(i32([1, 1, 1, 1, 1] if i % 3 else [1, 7, 40, 1, 1]))
        qkv.copy_(a.inputs())
        want = a.step(new, qkv)
        g.replay()
        assert all(torch.equal(s, t) for s, t in zip(want, got)), i
        assert all(torch.equal(s, t) for s, t in zip(a.state(), b.state())), i
    attn.query_status(a.status)
    attn.query_status(b.status)


def test_pages_and_rows_past_32_bits():
    """The same requests in the first pages of a cache of 9 GB and in its last ones, and
    with rows 4 GB apart: the same bits from each operator."""
    h, d, page, pages, lens = 8, 64, 256, 70000, [700, 530]
    c = kv.KV4Cache.empty(pages, h, d, d, page_size=page)
    tables = [[[3, 1, 2], [3, 1, 4]], [[pages - 1, pages - 3, pages - 2], [pages - 1, pages - 3, pages - 4]]]
    g = torch.Generator().manual_seed(23)
    k, v = (torch.randn(512 + 188 + 18, h, d, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(2, 1, 16, d, generator=g).to(BF).cuda()
    far = 2 ** 31 + 1024
    buf = torch.empty(far + 16 * d, dtype=BF, device="cuda")
    q_far = buf.as_strided(q.shape, (far, 16 * d, d, 1))
    q_far.copy_(q)
    n, starts, shared = i32(lens), i32([0, 2]), i32([512])
    got = []
    for i, t in enumerate(tables):
        at = [t[0][j // page] * page + j % page for j in range(700)] + [t[1][2] * page + j for j in range(18)]
        kv.kv4_write(c, k, v, i32(at))
        table, status = i32(t), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = q_far if i else None  # (q is not needed any more where o goes)
        o, lse = kv.kv4_decode_shared(q if i else q_far, c, table, n, starts, shared, out=out, status=status)
        w = kv.kv4_weights(q, c, table, n, lse, torch.zeros(2, h, 768, device="cuda"), status=status)
        before = w.clone()
        e = kv.kv4_evict(c, table, n, w, keep=525, first=i32([512, 512]), recent=4, status=status)
        attn.query_status(status)
        slots = i32([[t[b][j // page] * page + j % page for j in range(525)] for b in range(2)])
        got.append([o.clone(), lse, before, w, e.kept, e.seq_lens, *kv.kv4_read(c, slots.flatten())])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_positions_after_evictions_are_those_of_the_text():
    """The loop that kv's head describes, with budgets that are passed often: every row of the
    cache is what a cache without a budget holds at that token's place in the text, bit for bit."""
    b, hk, d, page, keep, steps = 4, 2, 64, 16, 40, 30
    g = torch.Generator().manual_seed(24)
    fresh = torch.randint(0, 6, (steps, b), generator=g).int()
    fresh[0] = torch.tensor([30, 45, 8, 0], dtype=torch.int32)
    rows = int(fresh.sum(1).max()) + 3
    total = fresh.sum(0)
    cos, sin = attn.rope_tables(int(total.max()), d)
    cache, table = empty_cache(40, hk, d, d, page), torch.full((b, 8), -1, dtype=torch.int32, device="cuda")
    free, status = torch.randperm(40, generator=g).int().cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    head, ctx, gone, first = i32([0]), i32([0] * b), i32([0] * b), i32([4, 0, 4, 2])
    w = torch.zeros(b, hk, 8 * page, device="cuda")
    row = torch.arange(rows, dtype=torch.int32, device="cuda")
    held = [[[] for _ in range(hk)] for _ in range(b)]  # places in the text of the tokens held
    text_k, text_v = [[] for _ in range(b)], [[] for _ in range(b)]
    for new in fresh:
        q, k, v = (torch.randn(rows, hk, d, generator=g).to(BF).cuda() for _ in range(3))
        p = kv.plan(ctx, new.cuda(), table, page_size=page, num_pages=40, rows=rows, free_pages=free, free_head=head,
                    status=status)
        request = torch.searchsorted(p.cu_seqlens[1:], row, right=True)
        positions = torch.where(p.positions < 0, -1, p.positions + gone[request.clamp(max=b - 1)])
        _, turned = attn.qk_norm_rope(q, k, cos, sin, positions=positions, status=status)
        kv.kv4_write(cache, turned, v, p.slots, status=status)
        w += torch.rand(w.shape, generator=g).cuda()
        r = kv.kv4_evict(cache, table, p.seq_lens, w, keep=keep, first=first, recent=3, free_pages=free,
                         free_head=p.free_head, status=status)
        gone += p.seq_lens - r.seq_lens
        head, ctx = r.free_head, r.seq_lens
        at, kept = 0, r.kept.tolist()
        for i, n in enumerate(new.tolist()):
            done = len(text_k[i])
            text_k[i] += list(k[at:at + n])
            text_v[i] += list(v[at:at + n])
            at += n
            for h in range(hk):
                places = held[i][h] + list(range(done, done + n))
                held[i][h] = [places[j] for j in kept[i][h] if j >= 0]
    attn.query_status(status)
    assert (total > keep).sum() >= 3 and gone.tolist() == (total - torch.tensor(ctx.tolist())).tolist()
    for i in range(b):
        n, m = len(text_k[i]), int(ctx[i])
        whole = empty_cache(n // page + 1, hk, d, d, page)
        k, v = torch.stack(text_k[i]), torch.stack(text_v[i])
        place = torch.arange(n, dtype=torch.int32, device="cuda")
        _, turned = attn.qk_norm_rope(k, k, cos, sin, positions=place)
        kv.kv4_write(whole, turned, v, place)
        want = kv.kv4_read(whole, place)
        t = table[i].tolist()
        got = kv.kv4_read(cache, i32([t[j // page] * page + j % page for j in range(m)]))
        for h in range(hk):
            for a, c in zip(got, want):
                assert torch.equal(a[:, h], c[torch.tensor(held[i][h]), h]), (i, h)
