"""The page plan, the 4-bit cache and attention over it, on the GPU, against the
float64 forms in kvref.py.

Plans and codes are whole numbers and must be equal.  Attention, from the
arithmetic (u: half a step of q's type): the result is rounded once, u |o|; a
probability times a scale is rounded once for the second product, u sum p |v|; a
score carries 2^-20 of sum |q k| (products are exact, at most 8 + 16 + 2 FP32
sums and scalings of 2^-23 at worst follow), which changes p by as much, as do
the base-2 exponentials (2^-21) and the sums over up to 2^10 tiles a warp
(2^-23 each with truncation: 2^-13 of sum p |v| at most, reached only by the
longest)."""
import math

import pytest
import torch

import kvref
from bwd_tcgen05_tmem_gb300 import attn, kv

pytestmark = pytest.mark.gpu
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bwd_tcgen05_tmem_gb300 import build
    build.build()
    attn.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan

def run_plan(ctx, new, page, cols, rows, seed=0, short=0, alloc=True):
    """A random table and free list; the kernel's plan against the lists'."""
    g = torch.Generator().manual_seed(seed)
    b = len(ctx)
    num = max(1, 2 * b * cols)
    perm = torch.randperm(num, generator=g).tolist()
    table = [[-7] * cols for _ in range(b)]
    at = 0
    for i in range(b):
        for j in range(-(-(ctx[i] if alloc else ctx[i] + new[i]) // page)):
            table[i][j] = perm[at]
            at += 1
    need = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new)) if alloc else 0
    free = [999999, 999998] + perm[at:at + need - short] if alloc else None
    t = i32(table) if b else torch.empty(0, cols, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(free_pages=i32(free), free_head=i32([2])) if alloc else {}
    got = kv.plan(i32(ctx), i32(new), t, page_size=page, num_pages=num, rows=rows, status=status, **kw)
    want = kvref.plan(ctx, new, table, page, num, rows, free, 2)
    torch.cuda.synchronize()
    assert got.cu_seqlens.tolist() == want[0]
    assert got.seq_lens.tolist() == want[1]
    assert got.positions.tolist() == want[2]
    assert got.slots.tolist() == want[3]
    assert t.tolist() == want[4]
    if alloc:
        assert got.free_head.tolist() == [want[5]]
    return status


@pytest.mark.parametrize("alloc", [True, False])
@pytest.mark.parametrize("b,page,most,new", [(1, 16, 1, 1), (1, 256, 5000, 700), (3, 64, 64, 64), (64, 64, 900, 1),
                                             (255, 32, 200, 40), (257, 16, 130, 9), (1030, 128, 300, 300)])
def test_plan(b, page, most, new, alloc):
    g = torch.Generator().manual_seed(b + page)
    ctx = torch.randint(0, most + 1, (b,), generator=g).tolist()
    fresh = torch.randint(0, new + 1, (b,), generator=g).tolist()
    fresh[-1] = 0
    cols = -(-(most + new) // page)
    status = run_plan(ctx, fresh, page, cols, sum(fresh) + 3, seed=b, alloc=alloc)
    attn.query_status(status)


def test_plan_borders():
    """Full and empty pages, requests of length 0, an exact fit, no rows, no requests."""
    for ctx, new in (([0, 16, 32, 15, 17], [16, 1, 0, 1, 15]), ([0, 0, 0], [0, 0, 0]), ([48], [0]), ([0], [48])):
        attn.query_status(run_plan(ctx, new, 16, 3, sum(new)))
    run_plan([], [], 16, 4, 5)
    run_plan([], [], 16, 4, 0, alloc=False)


def test_plan_largest_batch():
    b = 8192
    g = torch.Generator().manual_seed(1)
    ctx = torch.randint(0, 40, (b,), generator=g).tolist()
    new = torch.randint(0, 4, (b,), generator=g).tolist()
    attn.query_status(run_plan(ctx, new, 16, 3, sum(new) + 100))


def test_plan_reports_what_does_not_fit():
    for kw in (dict(rows=20), dict(rows=31, short=2)):
        rows = kw.pop("rows")
        status = run_plan([5, 30, 0], [20, 1, 10], 16, 2, rows, **kw)
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)


@pytest.mark.parametrize("ctx,new", [([-1, 5], [3, 2]), ([4, 5], [-3, 2]), ([33, 5], [0, 2]), ([30, 5], [3, 2]),
                                     ([2 ** 31 - 1, 5], [2 ** 31 - 1, 2])])
def test_plan_counts_requests_out_of_range_as_empty(ctx, new):
    t = i32([[0, 1], [2, 3]])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = kv.plan(i32(ctx), i32(new), t, page_size=16, num_pages=8, rows=6, free_pages=i32([5, 6, 7]),
                free_head=i32([0]), status=status)
    assert p.cu_seqlens.tolist() == [0, 0, 2] and p.seq_lens.tolist() == [0, 7]
    assert p.positions.tolist() == [5, 6, -1, -1, -1, -1] and p.slots.tolist() == [37, 38, -1, -1, -1, -1]
    assert t.tolist() == [[0, 1], [2, 3]] and p.free_head.tolist() == [0]
    with pytest.raises(attn.AttnError):
        attn.query_status(status)


def test_plan_does_not_use_bad_pages():
    t = i32([[100, -1], [2, 3]])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = kv.plan(i32([0, 0]), i32([20, 3]), t, page_size=16, num_pages=8, rows=23, status=status)
    assert p.slots.tolist() == [-1] * 20 + [32, 33, 34]
    p = kv.plan(i32([16, 0]), i32([4, 3]), t, page_size=16, num_pages=8, rows=7, status=status,
                free_pages=i32([8, -4, 1]), free_head=i32([-1]))
    assert p.slots.tolist() == [-1] * 7 and t.tolist() == [[100, -1], [-1, 3]]
    with pytest.raises(attn.AttnError):
        attn.query_status(status)


def test_plan_strided_table_and_given_outputs():
    wide = torch.full((3, 10), -3, dtype=torch.int32, device="cuda")
    t = wide[:, 2:6]
    out = kv.Plan(*(torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (4, 3, 12, 12, 1)))
    p = kv.plan(i32([0, 0, 0]), i32([5, 0, 3]), t, page_size=16, num_pages=9, rows=12, free_pages=i32([4, 8]),
                free_head=i32([0]), out=out)
    assert p is out and out.slots.tolist() == [64, 65, 66, 67, 68, 128, 129, 130] + [-1] * 4
    assert wide[:, 2].tolist() == [4, -3, 8] and (wide[:, [0, 1, 3, 4, 5, 6, 7, 8, 9]] == -3).all()


# ------------------------------------------------------------------ the cache

def empty_cache(pages, h, dqk, dv, page, fill=0xFF):
    c = kv.KV4Cache.empty(pages, h, dqk, dv, page_size=page)
    for t in (c.k_codes, c.v_codes):
        t.fill_(fill)
    for t in (c.k_scales, c.v_scales):
        t.fill_(float("nan"))
    return c


def specials(t, h, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, d, generator=g) * torch.exp2(torch.randint(-10, 11, (t, h, 1), generator=g).float())
    x = x.to(dt)
    if t > 8:
        tiny = torch.finfo(dt).smallest_normal
        x[1] = 0.0
        x[2, :, :32] = 0.0
        x[3, 0, 5] = float("inf")
        x[4, 0, 40] = float("nan")
        x[5] = (x[5].float() / x[5].float().abs().max() * tiny * 3).to(dt)  # below the normal range
        x[6] = (torch.randint(-14, 15, (h, d), generator=g) * 0.5).to(dt)   # scale 1: many ties
        x[6, :, ::32] = 7.0
        x[7] = (x[7].float() / x[7].float().abs().max() * torch.finfo(dt).max).to(dt)
    return x


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("t,h,dqk,dv,page", [(1, 1, 64, 64, 16), (13, 3, 128, 128, 32), (40, 8, 192, 128, 64),
                                             (257, 2, 256, 256, 128), (33, 1, 64, 64, 256), (700, 5, 128, 128, 16)])
def test_write_and_read(t, h, dqk, dv, page, dt):
    pages = -(-t // page) + 2
    cache = empty_cache(pages, h, dqk, dv, page)
    g = torch.Generator().manual_seed(t)
    k, v = specials(t, h, dqk, dt, t), specials(t, h, dv, dt, t + 1)
    slots = torch.randperm(pages * page, generator=g)[:t]
    out = torch.zeros(t, dtype=torch.bool)
    out[t // 2::5] = t > 1
    sl = torch.where(out, torch.tensor(-1), slots)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kv4_write(cache, k.cuda(), v.cuda(), sl.int().cuda(), status=status)
    torch.cuda.synchronize()
    live = ~out
    p, o = slots // page, slots % page
    for x, codes, scales, is_k in ((k, cache.k_codes, cache.k_scales, True), (v, cache.v_codes, cache.v_scales, False)):
        c, s = kvref.quantise(x.double())
        codes, scales = codes.cpu(), scales.cpu()
        assert torch.equal(codes[p, :, o][live], kvref.pack(c, is_k)[live])
        got = scales[p, :, o][live].double()
        want = s[live]
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
        rest = torch.ones(pages, page, dtype=torch.bool)
        rest[p[live], o[live]] = False
        assert (codes.transpose(1, 2)[rest] == 0xFF).all() and torch.isnan(scales.transpose(1, 2)[rest].float()).all()
    rk, rv = (torch.full((t, h, d), 7.0, dtype=dt, device="cuda") for d in (dqk, dv))
    kv.kv4_read(cache, sl.int().cuda(), k=rk, v=rv, status=status)
    attn.query_status(status)
    for x, r in ((k, rk), (v, rv)):
        want = kvref.values(*kvref.quantise(x.double())).to(dt)
        r = r.cpu()
        assert torch.equal(torch.isnan(r[live]), torch.isnan(want[live]))
        assert torch.equal(r[live].nan_to_num(), want[live].nan_to_num())
        assert (r[out] == 7.0).all()


def test_write_and_read_strided_and_out_of_range():
    cache = empty_cache(3, 2, 128, 128, 16)
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(9, 8, 128, generator=g).to(BF).cuda()
    k, v = qkv[:, 4:6], qkv[:, 6:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kv4_write(cache, k, v, i32([3, 4, 47, 0, 1, 2, 40, 41, 42]), status=status)
    attn.query_status(status)
    buf = torch.full((9, 8, 128), 5.0, dtype=BF, device="cuda")
    before = [t.clone() for t in (cache.k_codes, cache.v_codes)]
    kv.kv4_read(cache, i32([3, 4, 47, 0, 1, 2, 48, 41, 2 ** 31 - 1]), k=buf[:, 2:4], v=buf[:, 5:7], status=status)
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)
    want = [kvref.values(*kvref.quantise(t.cpu().double())).to(BF) for t in (k, v)]
    for a, w in ((buf[:, 2:4], want[0]), (buf[:, 5:7], want[1])):
        a = a.cpu()
        assert torch.equal(a[[0, 1, 2, 3, 4, 5, 7]], w[[0, 1, 2, 3, 4, 5, 7]]) and (a[[6, 8]] == 5.0).all()
    assert (buf[:, [0, 1, 4, 7]] == 5.0).all()
    status.zero_()
    kv.kv4_write(cache, k, v, i32([48, 49, 5000, 2 ** 31 - 1, -1, -2, 48, 48, 48]), status=status)
    with pytest.raises(attn.AttnError):
        attn.query_status(status)
    assert torch.equal(before[0], cache.k_codes) and torch.equal(before[1], cache.v_codes)


# ------------------------------------------------------------------ attention

class Held:
    """Random sequences of given lengths in a cache whose other bytes are
    poison: codes 0xFF, scales NaN, table entries out of range."""

    def __init__(self, lens, h, dqk, dv, page, dt, seed, vscale=1.0, cols=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.dt = list(lens), page, dt
        need = [-(-n // page) for n in lens]
        cols = cols or max(1, max(need, default=0)) + 1
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g).tolist()
        self.table, at = [], 0
        for n in need:
            self.table.append(perm[at:at + n] + [(-5, 10 ** 9)[i % 2] for i in range(cols - n)])
            at += n
        self.cache = empty_cache(pages, h, dqk, dv, page)
        total = sum(lens)
        self.k = torch.randn(total, h, dqk, generator=g).to(dt)
        self.v = (torch.randn(total, h, dv, generator=g) * vscale).to(dt)
        slots = [self.table[b][j // page] * page + j % page for b, n in enumerate(lens) for j in range(n)]
        if total:
            kv.kv4_write(self.cache, self.k.cuda(), self.v.cuda(), i32(slots))
        self.slots = slots
        self.t, self.l = i32(self.table) if len(lens) else torch.empty(0, cols, dtype=torch.int32, device="cuda"), i32(self.lens)
        self.g = g

    def q(self, sq, hq, scale=1.5):
        d = self.cache.d_qk
        return (torch.randn(len(self.lens), sq, hq, d, generator=self.g) * scale).to(self.dt).cuda()

    def reference(self, q, **kw):
        c = self.cache
        dev = "cuda"
        kc, vc = kvref.unpack(c.k_codes, True).to(dev), kvref.unpack(c.v_codes, False).to(dev)
        safe = [[p if 0 <= p < c.num_pages else 0 for p in r] for r in self.table]
        return kvref.decode(q.double(), kc, c.k_scales.double(), vc, c.v_scales.double(), safe, self.lens,
                            kw.pop("scale", 1 / math.sqrt(c.d_qk)), **kw)

    def check(self, q, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = kv.kv4_decode(q, self.cache, self.t, self.l, status=status, **kw)
        o2, lse2 = kv.kv4_decode(q, self.cache, self.t, self.l, **kw)
        attn.query_status(status)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        kw.pop("o_dtype", None)
        within(o, lse, self.reference(q, **kw), UNIT[self.dt])
        return o, lse


def within(o, lse, ref, u):
    ro, rl, mag, big = ref
    assert torch.isfinite(o).all()
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o[empty.transpose(1, 2)] == 0).all()
    score = 2.0 ** -20 * big
    err = (lse.double() - rl)[~empty].abs()
    assert (err <= score[~empty] + 2.0 ** -21 * rl[~empty].abs() + 2.0 ** -19).all(), float(err.max())
    out = u if o.dtype != torch.float32 else 0.0
    tol = out * ro.abs() + (u + 2.0 ** -13) * mag + score.transpose(1, 2)[..., None] * mag + 2.0 ** -25
    err = (o.double() - ro).abs()
    assert (err <= tol).all(), (float((err - tol).max()), float((err / tol).max()))


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 256, 257, 300, 511, 513, 1000]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("dqk,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("hkv,group,sq,page", [(2, 4, 1, 64), (1, 1, 3, 16), (2, 8, 2, 32), (3, 5, 1, 128)])
def test_decode(dqk, dv, hkv, group, sq, page, dt):
    x = Held(LENS, hkv, dqk, dv, page, dt, seed=dqk + group)
    x.check(x.q(sq, hkv * group))


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 1), (5, 0), (31, 4), (32, 32), (40, 33), (100, 700), (255, 64), (2000, 3),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("page,sq", [(16, 1), (64, 4), (256, 2)])
def test_decode_window_and_sinks(window, sinks, page, sq):
    x = Held(LENS, 2, 128, 128, page, BF, seed=window % 1000 + sinks % 1000)
    x.check(x.q(sq, 8), window_left=window, sinks=sinks)


@pytest.mark.parametrize("sq,hkv,group", [(1, 1, 128), (17, 2, 3), (64, 1, 8), (256, 1, 2), (1, 16, 1), (5, 2, 12)])
def test_decode_rows(sq, hkv, group):
    x = Held([0, 3, 70, 300, 256], hkv, 128, 128, 64, BF, seed=sq + group)
    x.check(x.q(sq, hkv * group))
    x.check(x.q(sq, hkv * group), window_left=50, sinks=10)


@pytest.mark.parametrize("lens", [[50000], [1], [20000, 1, 0, 7, 9000], [33] * 300, list(range(0, 600))])
def test_decode_batches(lens):
    """One long sequence cut over all blocks; ragged ones; more sequences than threads."""
    x = Held(lens, 2, 64, 64, 64, BF, seed=len(lens))
    x.check(x.q(1, 8))


@pytest.mark.parametrize("vscale", [1e-4, 1e-2, 1000.0])
def test_decode_small_and_large_values(vscale):
    """fp16 probabilities times scales stay in range whatever the size of V, and
    a few tokens much larger than the others do not take their precision."""
    x = Held([700, 40], 2, 128, 128, 64, FP, seed=3, vscale=vscale)
    x.check(x.q(1, 8))
    x.check(x.q(1, 8, scale=20.0))  # a sharp softmax


def test_decode_scale_and_fp32_output():
    x = Held([300, 77], 2, 128, 128, 32, BF, seed=4)
    x.check(x.q(2, 6), scale=0.3)
    x.check(x.q(2, 6), o_dtype=torch.float32)


def test_decode_nan_reaches_the_rows_that_see_it_only():
    x = Held([100, 100], 2, 128, 128, 32, BF, seed=6)
    q = x.q(3, 4)
    clean = kv.kv4_decode(q, x.cache, x.t, x.l)
    p = x.table[0][98 // 32]
    for t, at in ((x.cache.v_scales, 2), (x.cache.k_scales, 1)):
        held = t.clone()
        t[p, 1, 98 % 32, at] = float("nan")  # token 98 of kv head 1: queries 1 and 2 see it
        o, lse = kv.kv4_decode(q, x.cache, x.t, x.l)
        assert torch.equal(o[1], clean[0][1]) and torch.equal(o[0, :, :2], clean[0][0, :, :2])
        assert torch.equal(o[0, 0], clean[0][0, 0]) and torch.equal(lse[0, :, 0], clean[1][0, :, 0])
        hit = o[0, 1:, 2:]
        assert torch.isnan(hit[..., 64:96]).all()
        if t is x.cache.k_scales:
            assert torch.isnan(hit).all() and torch.isnan(lse[0, 2:, 1:]).all()
        else:
            assert torch.isfinite(hit[..., :64]).all() and torch.isfinite(hit[..., 96:]).all()
        # a window that leaves it out
        o, lse = kv.kv4_decode(q[:, 2:], x.cache, x.t, x.l, window_left=0)
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        t.copy_(held)


def test_decode_strided_and_other_stream():
    x = Held([300, 5, 77], 2, 128, 128, 64, BF, seed=7)
    q = x.q(2, 8)
    want = kv.kv4_decode(q, x.cache, x.t, x.l)
    wide = torch.zeros(3, 2, 12, 136, dtype=BF, device="cuda")
    wide[:, :, 2:10, :128] = q
    out = torch.full((3, 8, 2, 136), 9.0, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    table = torch.cat((torch.full_like(x.t, -1), x.t), 1)[:, x.t.shape[1]:]
    kv.kv4_decode(wide[:, :, 2:10, :128], x.cache, table, x.l, out=out.transpose(1, 2)[..., 8:], stream=side)
    side.synchronize()
    assert torch.equal(out.transpose(1, 2)[..., 8:], want[0]) and (out[..., :8] == 9.0).all()


def test_decode_lengths_and_pages_out_of_range():
    x = Held([100, 100, 100], 2, 128, 128, 32, BF, seed=8)
    q = x.q(1, 4)
    clean, _ = kv.kv4_decode(q, x.cache, x.t, x.l)
    for bad in (-1, x.t.shape[1] * 32 + 1, 2 ** 31 - 1, -2 ** 31):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = kv.kv4_decode(q, x.cache, x.t, i32([100, bad, 100]), status=status)
        assert (o[1] == 0).all() and torch.isneginf(lse[1]).all() and torch.equal(o[[0, 2]], clean[[0, 2]])
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
    t = x.t.clone()
    t[1, 1], t[1, 2] = -1, 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, _ = kv.kv4_decode(q, x.cache, t, x.l, status=status)
    assert torch.equal(o[[0, 2]], clean[[0, 2]])
    with pytest.raises(attn.AttnError):
        attn.query_status(status)


def test_decode_offsets_past_32_bits():
    """A cache whose codes take more than 4 GiB a side: pages at both ends."""
    h, page, pages = 8, 256, 40000
    cache = kv.KV4Cache.empty(pages, h, 128, 128, page_size=page)
    assert cache.k_codes.numel() > 2 ** 32
    small = Held([500, 300], h, 128, 128, page, BF, seed=9)
    q = small.q(1, 16)
    want = kv.kv4_decode(q, small.cache, small.t, small.l)
    far = [pages - 1, 0, pages - 2, 7]
    table = i32([[far[0], far[1]], [far[2], far[3]]])
    slots = [(far[2 * b + j // page]) * page + j % page for b, n in ((0, 500), (1, 300)) for j in range(n)]
    kv.kv4_write(cache, small.k.cuda(), small.v.cuda(), i32(slots))
    got = kv.kv4_decode(q, cache, table, small.l)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = kv.kv4_read(cache, i32(slots)), kv.kv4_read(small.cache, i32(small.slots))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_captured_with_other_lengths_and_a_shared_workspace():
    """One graph serves any lengths; two graphs that share a workspace, replayed
    one after the other, do not disturb each other."""
    x = Held([700, 40, 0, 1], 2, 128, 128, 64, BF, seed=10)
    q = [x.q(1, 8), x.q(3, 8)]
    ws = torch.empty(max(kv.decode_workspace_size(t, x.cache, x.t) for t in q), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    lens = x.l.clone()
    outs, graphs = [], []
    for t in q:
        kv.kv4_decode(t, x.cache, x.t, lens, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(kv.kv4_decode(t, x.cache, x.t, lens, workspace=ws))
    for other in ([700, 40, 0, 1], [3, 0, 0, 1], [650, 39, 0, 0], [0, 0, 0, 0], [257, 40, 0, 1]):
        lens.copy_(i32(other))
        for rep in range(2):
            for gr in graphs:
                gr.replay()
        torch.cuda.synchronize()
        for t, got in zip(q, outs):
            want = kv.kv4_decode(t, x.cache, x.t, i32(other))
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_empty_batch_and_partial_results_merge():
    x = Held([], 2, 128, 128, 64, BF, seed=11)
    o, lse = kv.kv4_decode(torch.empty(0, 1, 4, 128, dtype=BF, device="cuda"), x.cache, x.t, x.l)
    assert o.shape == (0, 1, 4, 128)
    # two halves of a context, merged by attn_lse_merge, are the whole
    x = Held([512], 2, 128, 128, 64, BF, seed=12)
    q = x.q(1, 8)
    whole, lse = kv.kv4_decode(q, x.cache, x.t, x.l, o_dtype=torch.float32)
    parts = [kv.kv4_decode(q, x.cache, t.contiguous(), i32([256]), o_dtype=torch.float32)
             for t in (x.t[:, :4], x.t[:, 4:8])]
    m, ml = attn.lse_merge([p[0][0].contiguous() for p in parts], [p[1][0] for p in parts], [0, 0], [1, 1], 1,
                           out_dtype=torch.float32)
    ref = x.reference(q)
    within(m[None], ml[None], ref, UNIT[BF])


def test_decode_one_long_and_many_short_requests():
    """Cut by runs: an item that many runs share among hundreds that none do."""
    x = Held([30000] + [21] * 500 + [9000], 2, 64, 64, 64, FP, seed=13)
    x.check(x.q(1, 4))
    x.check(x.q(3, 8))


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-6])
def test_decode_tiny_scale_is_a_mean(scale):
    """Hidden tokens stay hidden where every score is next to nothing."""
    x = Held([70, 5, 0, 130], 2, 128, 128, 64, BF, seed=14)
    x.check(x.q(3, 8, scale=0.0), scale=scale)
    x.check(x.q(3, 8), scale=scale, window_left=9, sinks=2)


def test_decode_hidden_scales_may_be_infinite():
    x = Held([200, 64], 2, 128, 128, 64, BF, seed=15)
    q = x.q(4, 4)
    want = kv.kv4_decode(q, x.cache, x.t, x.l, window_left=20, sinks=3)
    for j in (3, 100, 175):  # no query sees these
        x.cache.v_scales[x.table[0][j // 64], :, j % 64] = float("inf")
        x.cache.k_scales[x.table[0][j // 64], :, j % 64] = float("-inf")
    got = kv.kv4_decode(q, x.cache, x.t, x.l, window_left=20, sinks=3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x.cache.v_scales[x.table[0][199 // 64], :, 199 % 64] = float("inf")  # the last query alone
    got = kv.kv4_decode(q, x.cache, x.t, x.l, window_left=20, sinks=3)
    assert torch.equal(got[0][:, :3], want[0][:, :3]) and torch.equal(got[0][1], want[0][1])
    assert not torch.isfinite(got[0][0, 3]).any()


def test_decode_two_streams_at_once():
    x = [Held([3000, 40, 900], 2, 128, 128, 64, BF, seed=16), Held([5000], 4, 64, 64, 32, FP, seed=17)]
    q = [x[0].q(1, 8), x[1].q(2, 8)]
    want = [kv.kv4_decode(a, y.cache, y.t, y.l) for a, y in zip(q, x)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(kv.kv4_decode(q[i], x[i].cache, x[i].t, x[i].l))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


# ------------------------------------------------------------------ together

def test_serving_steps():
    """plan, norm + rotation, write, attend: a prompt, then steps of ragged
    batches, against float64 attention over the quantised rows."""
    hq, hk, d, page, b = 8, 2, 128, 32, 4
    g = torch.Generator().manual_seed(13)
    cos, sin = attn.rope_tables(512, d)
    w = (1 + 0.2 * torch.randn(2, d, generator=g)).cuda()
    cache = empty_cache(64, hk, d, d, page)
    table = torch.full((b, 8), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(64, generator=g).int().cuda(), i32([0])
    ctx = i32([0] * b)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = Held([0] * b, hk, d, d, page, BF, seed=14)  # for its reference
    x.cache = cache
    for new in ([70, 1, 0, 129], [1, 1, 1, 1], [1, 1, 1, 1], [1, 0, 1, 1]):
        rows = sum(new) + 2
        qkv = torch.randn(rows, hq + 2 * hk, d, generator=g).to(BF).cuda()
        p = kv.plan(ctx, i32(new), table, page_size=page, num_pages=64, rows=rows, free_pages=free, free_head=head,
                    status=status)
        q, k = attn.qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], cos, sin, positions=p.positions, wq=w[0], wk=w[1],
                                 status=status)
        kv.kv4_write(cache, k, qkv[:, hq + hk:], p.slots, status=status)
        ctx, head = p.seq_lens, p.free_head
        if max(new) > 1:
            continue
        # one query for each request; those without a new token ask again with their last row
        last = (p.cu_seqlens[1:].long() - 1).clamp(min=0)
        qs = q[last][:, None]
        o, lse = kv.kv4_decode(qs, cache, table, ctx, status=status)
        x.lens, x.table = ctx.tolist(), table.tolist()
        within(o, lse, x.reference(qs), UNIT[BF])
    attn.query_status(status)
    assert ctx.tolist() == [73, 3, 3, 132] and head.tolist() == [3 + 1 + 1 + 5]


def test_prompt_chunk_over_a_cached_prefix():
    """plan (map only), read, attn.fwd bottom-right: the attention of a chunk,
    equal to attention over the cache within both bounds."""
    x = Held([200], 2, 128, 128, 64, BF, seed=15)
    q = x.q(16, 4)
    p = kv.plan(i32([0]), x.l, x.t, page_size=64, num_pages=x.cache.num_pages, rows=200)
    assert p.slots.tolist() == x.slots
    k, v = kv.kv4_read(x.cache, p.slots)
    o, lse = attn.fwd(q, k[None], v[None], causal=True, bottom_right=True)
    ro, rl, mag, big = x.reference(q)
    # k and v are rounded to bf16 on the way (the codes times their scale have 11 bits)
    u = UNIT[BF]
    assert ((lse.double() - rl).abs() <= u * big + 1e-4).all()
    assert ((o.double() - ro).abs() <= u * ro.abs() + (2 * u + 2.0 ** -12) * mag + 2 * u * big.transpose(1, 2)[..., None] * mag).all()
    o2, lse2 = kv.kv4_decode(q, x.cache, x.t, x.l)
    within(o2, lse2, (ro, rl, mag, big), u)


def test_plan_with_an_empty_free_list():
    """No page is left: tokens past the held pages get none, whatever the table
    holds there; without need of a page the head passes through."""
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    for free in (none, i32([4, 5])[2:]):
        t = i32([[3, 5], [2, 1]])  # (entries 5 and 1 are valid pages that are not held)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        p = kv.plan(i32([10, 16]), i32([10, 1]), t, page_size=16, num_pages=8, rows=12, free_pages=free,
                    free_head=i32([4]), status=status)
        assert p.positions.tolist() == list(range(10, 20)) + [16, -1]
        assert p.slots.tolist() == list(range(58, 64)) + [-1] * 6
        assert t.tolist() == [[3, -1], [2, -1]] and p.free_head.tolist() == [6]
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
        t = i32([[3, 5]])
        status.zero_()
        p = kv.plan(i32([10]), i32([6]), t, page_size=16, num_pages=8, rows=6, free_pages=free, free_head=i32([0]),
                    status=status)
        assert p.slots.tolist() == list(range(58, 64)) and t.tolist() == [[3, 5]] and p.free_head.tolist() == [0]
        attn.query_status(status)


@pytest.mark.parametrize("power", [40, 50, 70, 95])
@pytest.mark.parametrize("n", [200, 300000])
def test_decode_large_values_after_empty_ones(n, power):
    """Tiles of 64 tokens whose V is zero, before and between tiles of values of
    about 2^power: the sum and the LSE keep all of their tokens.  n = 300000 gives
    a warp two tiles; with n = 200 the join meets the pieces."""
    x = Held([n], 1, 64, 64, 64, BF, seed=18)
    at = torch.arange(n)
    pages = torch.tensor(x.table[0])[at // 64]
    even = at // 64 % 2 == 0
    x.cache.v_scales[pages[even], :, at[even] % 64] = 0.0
    odd = (pages[~even].cuda(), slice(None), at[~even].cuda() % 64)
    x.cache.v_scales[odd] = x.cache.v_scales[odd] * 2.0 ** power
    x.check(x.q(1, 4))
    x.check(x.q(3, 4), o_dtype=torch.float32)


def test_plan_from_several_threads():
    """Batches that need different amounts of shared memory, planned at once.
    (Packed calls, so that the threads meet within the library.)"""
    import threading
    lib, failed = attn.fast(), []
    batches = [8192, 3500] * 4
    jobs = []
    for b in batches:
        t = [i32([0] * b), i32([1] * b), torch.zeros(b, 1, dtype=torch.int32, device="cuda")]
        out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (b + 1, b, 1, 1)]
        jobs.append((b, t, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(b, t, out, stream):
        p = attn._PLAN_PACK(b, 1, 16, 1, 1, 0, 1)
        args = (p, *(x.data_ptr() for x in t), None, None, *(x.data_ptr() for x in out), None, None,
                stream.cuda_stream)
        start.wait()
        for _ in range(300):
            rc = lib.attn_kv_plan(*args)
            if rc:
                failed.append((b, rc))
                return

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for b, _, out, _ in jobs:
        assert out[0].tolist() == list(range(b + 1)) and out[1].tolist() == [1] * b


def test_plan_with_as_many_rows_as_an_int_counts():
    """rows = 2^31 - 1: the loops' last steps pass that, and nothing lands before
    the arrays."""
    rows, guard = 2 ** 31 - 1, 1 << 20
    if torch.cuda.mem_get_info()[0] < 2 * (rows + guard) * 4 + (8 << 30):
        pytest.skip("needs 17 GB")
    whole = torch.full((2, rows + guard), 77, dtype=torch.int32, device="cuda")
    out = kv.Plan(i32([0, 0, 0]), i32([0, 0]), whole[0, guard:], whole[1, guard:], None)
    kv.plan(i32([5, 0]), i32([2, 3]), i32([[1], [4]]), page_size=16, num_pages=8, rows=rows, out=out)
    assert out.positions[:5].tolist() == [5, 6, 0, 1, 2] and out.slots[:5].tolist() == [21, 22, 64, 65, 66]
    for t in out[2:4]:
        lo, hi = torch.aminmax(t[5:])
        assert lo == -1 and hi == -1
    assert (whole[:, :guard] == 77).all()


@pytest.mark.parametrize("page", [16, 32])
def test_decode_pages_behind_the_window_may_be_gone(page):
    """Pages all of whose tokens lie before the window and after the first tokens
    are not looked at, also where they share a tile with visible ones."""
    x = Held([500, 333, 64, 17], 2, 128, 128, page, BF, seed=19)
    for sq, window, sinks in ((1, 20, 0), (3, 70, 5), (2, 100, 40), (1, 0, 1), (4, 130, 64)):
        q = x.q(sq, 8)
        want = kv.kv4_decode(q, x.cache, x.t, x.l, window_left=window, sinks=sinks)
        gone = x.t.clone()
        for b, n in enumerate(x.lens):
            for j in range(-(-n // page)):
                if (j + 1) * page <= n - sq - window and j * page >= sinks:
                    gone[b, j] = (-1, 2 ** 31 - 1)[j % 2]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = kv.kv4_decode(q, x.cache, gone, x.l, window_left=window, sinks=sinks, status=status)
        attn.query_status(status)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        if window:  # the first page that is needed
            need = max(0, 500 - sq - window) // page
            gone[0, need] = -1
            kv.kv4_decode(q, x.cache, gone, x.l, window_left=window, sinks=sinks, status=status)
            with pytest.raises(attn.AttnError, match="out of range"):
                attn.query_status(status)


def within_11_bits(o, lse, ref, dt):
    """within, with the second product's operand as the kernel holds it: fp16, half
    a step 2^-11, whatever q's type; only the result is rounded to ``dt``."""
    ro, rl, mag, big = ref
    score = 2.0 ** -20 * big
    out = UNIT[dt] if o.dtype != torch.float32 else 0.0
    tol = out * ro.abs() + (2.0 ** -11 + 2.0 ** -13) * mag + score.transpose(1, 2)[..., None] * mag + 2.0 ** -25
    err = (o.double() - ro).abs()
    assert torch.isfinite(o).all() and (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("o_dtype", [BF, torch.float32])
@pytest.mark.parametrize("dqk,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("group,sq,page,kw", [(4, 1, 64, {}), (8, 2, 16, {}), (5, 3, 32, dict(window_left=40, sinks=33)),
                                              (2, 1, 256, dict(window_left=255, sinks=4))])
def test_decode_probabilities_have_11_bits(dqk, dv, group, sq, page, kw, o_dtype):
    x = Held(LENS + [5000], 2, dqk, dv, page, BF, seed=20)
    q = x.q(sq, 2 * group)
    o, lse = kv.kv4_decode(q, x.cache, x.t, x.l, o_dtype=o_dtype, **kw)
    ref = x.reference(q, **kw)
    within(o, lse, ref, UNIT[BF])
    within_11_bits(o, lse, ref, BF)


def test_decode_probabilities_have_11_bits_in_large_batches():
    for lens in ([33] * 300, list(range(0, 600)), [30000] + [21] * 200):
        x = Held(lens, 2, 64, 64, 64, BF, seed=21)
        q = x.q(1, 8)
        o, lse = kv.kv4_decode(q, x.cache, x.t, x.l, o_dtype=torch.float32)
        within_11_bits(o, lse, x.reference(q), BF)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("dqk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("scale", [1.5, 6.0])
def test_decode_scores_of_few_tokens(dqk, dv, scale, dt):
    """The LSE of one to twenty tokens is a score or nearly one: nothing averages the
    products' sums out."""
    for seed in range(6):
        x = Held([1, 2, 3, 5, 9, 20] * 8, 3, dqk, dv, 64, dt, seed=seed)
        x.check(x.q(1, 24, scale=scale))
