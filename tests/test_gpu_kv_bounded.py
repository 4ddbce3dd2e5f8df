"""The weights that cached tokens receive, and eviction, on the GPU, against the
float64 forms in boundedref.py.

Weights, from the arithmetic: a score carries 2^-20 of sum |q k| (as in attention
over the cache), which changes its exponential by as much; the argument of the
base-2 exponential, x / ln 2 - LSE / ln 2, is rounded from factors rounded to 2^-24
each, so it carries 4 * 2^-24 of |x| + |LSE|, below 2^-21 (sum |q k| + |LSE|), and the
exponential 2^-21; then come sums of the rows and of the earlier entry, 2^-24 each of
what they hold.  Eviction moves bits: everything must be equal."""
import math

import pytest
import torch

import boundedref
import kvref
from bwd_tcgen05_tmem_gb300 import attn, kv
from test_gpu_kv import BF, FP, LENS, Held, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bwd_tcgen05_tmem_gb300 import build
    build.build()
    attn.load()


def zero():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ weights

def reference(x, q, lse, **kw):
    c = x.cache
    safe = [[p if 0 <= p < c.num_pages else 0 for p in r] for r in x.table]
    return boundedref.weights(q.double(), kvref.unpack(c.k_codes, True).cuda(), c.k_scales.double(), safe, x.lens,
                              lse, kw.pop("scale", 1 / math.sqrt(c.d_qk)), **kw)


def check_weights(x, q, capacity=None, **kw):
    """Both ways of writing, from entries that hold other numbers, against the reference."""
    lse = kv.kv4_decode(q, x.cache, x.t, x.l, **kw)[1]
    want = reference(x, q, lse, **kw)
    b, h = len(x.lens), x.cache.heads_kv
    cap = capacity or max(x.lens, default=0) + 5
    sq, rows = q.shape[1], q.shape[1] * q.shape[2] // h
    for add in (True, False):
        held = torch.rand(b, h, cap, generator=x.g).cuda() * 3
        w, status = held.clone(), zero()
        got = kv.kv4_weights(q, x.cache, x.t, x.l, lse, w, accumulate=add, status=status, **kw)
        assert got is w
        again = kv.kv4_weights(q, x.cache, x.t, x.l, lse, held.clone(), accumulate=add, **kw)
        attn.query_status(status)
        assert torch.equal(w, again)
        for i, n in enumerate(x.lens):
            assert torch.equal(w[i, :, n:], held[i, :, n:])
            ref, big, top = want[i]
            old = held[i, :, :n].double().clone()
            old[:, max(n - sq, 0):] = 0.0
            if not add:
                old[:] = 0.0
            tol = ref * (2.0 ** -20 * big + 2.0 ** -21 * (big + top) + 2.0 ** -21 + rows * 2.0 ** -24)
            tol += (old + ref) * 2.0 ** -23 + rows * 2.0 ** -120
            err = (w[i, :, :n].double() - old - ref).abs()
            assert (err <= tol).all(), (i, float((err / tol).max()))
    return lse


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("dqk,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("hkv,group,sq,page", [(2, 4, 1, 64), (1, 1, 3, 16), (2, 8, 2, 32), (3, 5, 1, 128),
                                               (2, 6, 7, 256)])
def test_weights(dqk, dv, hkv, group, sq, page, dt):
    x = Held(LENS, hkv, dqk, dv, page, dt, seed=dqk + group)
    check_weights(x, x.q(sq, hkv * group))


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 1), (5, 0), (31, 4), (100, 700), (255, 64), (2 ** 31 - 1, 3)])
@pytest.mark.parametrize("page,sq,group", [(16, 1, 4), (64, 4, 4), (256, 2, 1), (32, 40, 2)])
def test_weights_window_and_first_tokens(window, sinks, page, sq, group):
    x = Held(LENS, 2, 128, 128, page, BF, seed=window % 1000 + sinks)
    check_weights(x, x.q(sq, 2 * group), window_left=window, sinks=sinks)


@pytest.mark.parametrize("sq,hkv,group", [(1, 1, 128), (17, 2, 3), (64, 1, 8), (256, 1, 2), (1, 16, 1), (9, 2, 12)])
def test_weights_of_many_rows(sq, hkv, group):
    x = Held([0, 3, 70, 300, 256], hkv, 128, 128, 64, BF, seed=sq + group)
    check_weights(x, x.q(sq, hkv * group))
    check_weights(x, x.q(sq, hkv * group), window_left=50, sinks=10)


@pytest.mark.parametrize("lens", [[50000], [1], [20000, 1, 0, 7, 9000], [33] * 300, list(range(0, 600)), [0, 0, 0]])
def test_weights_of_batches(lens):
    x = Held(lens, 2, 64, 64, 64, BF, seed=len(lens))
    check_weights(x, x.q(1, 8))


def test_weights_sum_up_to_the_query_heads():
    """Each query head hands out 1."""
    x = Held([700, 1, 64], 2, 128, 128, 64, BF, seed=5)
    q = x.q(3, 8)
    lse = kv.kv4_decode(q, x.cache, x.t, x.l)[1]
    w = torch.full((3, 2, 704), float("nan"), device="cuda")
    kv.kv4_weights(q, x.cache, x.t, x.l, lse, w, accumulate=False)
    for i, n in enumerate(x.lens):
        seen = 4.0 * min(n, 3)  # queries at negative positions see nothing
        assert torch.allclose(w[i, :, :n].double().sum(-1), torch.full((2,), seen, dtype=torch.float64, device="cuda"),
                              atol=seen * 2.0 ** -14)


def test_weights_scale_and_large_queries():
    x = Held([300, 77], 2, 128, 128, 32, BF, seed=4)
    check_weights(x, x.q(2, 6), scale=0.3)
    check_weights(x, x.q(1, 6, scale=30.0))
    check_weights(x, x.q(1, 6, scale=1e-12))


def test_weights_strided_and_other_stream():
    x = Held([130, 64, 250], 2, 128, 128, 64, FP, seed=8)
    wide = torch.randn(3, 12, 2, 128, generator=x.g).to(FP).cuda()
    q = wide[:, 2:10].transpose(1, 2)
    lse = kv.kv4_decode(q, x.cache, x.t, x.l)[1]
    plain = kv.kv4_weights(q, x.cache, x.t, x.l, lse, torch.ones(3, 2, 260, device="cuda"))
    buf = torch.ones(2, 3, 300, device="cuda")
    w = buf.transpose(0, 1)[..., 7:267]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kv.kv4_weights(q, x.cache, x.t, x.l, lse, w, stream=s)
    s.synchronize()
    assert torch.equal(w, plain)
    assert (buf[..., :7] == 1).all() and (buf[..., 267:] == 1).all()


def test_weights_lengths_and_pages_out_of_range():
    x = Held([100, 50, 64], 2, 64, 64, 16, BF, seed=9)
    q = x.q(1, 4)
    lse = kv.kv4_decode(q, x.cache, x.t, x.l)[1]
    ones = torch.ones(3, 2, 112, device="cuda")
    good = kv.kv4_weights(q, x.cache, x.t, x.l, lse, ones.clone())
    for bad in (-1, 113, 2 ** 31 - 1):
        status = zero()
        got = kv.kv4_weights(q, x.cache, x.t, i32([100, bad, 64]), lse, ones.clone(), status=status)
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2]) and (got[1] == 1).all()
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
    # a row shorter than its sequence
    status = zero()
    got = kv.kv4_weights(q, x.cache, x.t, x.l, lse, ones[..., :64].clone(), status=status)
    assert (got[0] == 1).all() and torch.equal(got[2], good[2, :, :64])
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)
    t = x.t.clone()
    t[1, 1] = x.cache.num_pages
    status = zero()
    got = kv.kv4_weights(q, x.cache, t, x.l, lse, ones.clone(), status=status)
    assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)


def test_weights_pages_behind_the_window_may_be_gone():
    x = Held([900], 2, 128, 128, 16, BF, seed=10)
    q = x.q(2, 8)
    kw = dict(window_left=40, sinks=5)
    lse = kv.kv4_decode(q, x.cache, x.t, x.l, **kw)[1]
    w = torch.ones(1, 2, 900, device="cuda")
    whole = kv.kv4_weights(q, x.cache, x.t, x.l, lse, w.clone(), **kw)
    t, status = x.t.clone(), zero()
    t[0, 1:(900 - 2 - 40) // 16] = -1
    assert torch.equal(kv.kv4_weights(q, x.cache, t, x.l, lse, w.clone(), status=status, **kw), whole)
    attn.query_status(status)


def test_weights_nan_stays_with_its_token():
    x = Held([200, 200], 2, 128, 128, 64, BF, seed=11)
    q = x.q(1, 8)
    lse = kv.kv4_decode(q, x.cache, x.t, x.l)[1]
    w = kv.kv4_weights(q, x.cache, x.t, x.l, lse, torch.ones(2, 2, 200, device="cuda"))
    x.cache.k_scales[x.table[0][1], 1, 7, 2] = float("nan")
    got = kv.kv4_weights(q, x.cache, x.t, x.l, lse, torch.ones(2, 2, 200, device="cuda"))
    bad = torch.isnan(got)
    assert bad[0, 1, 71] and int(bad.sum()) == 1
    assert torch.equal(got[~bad], w[~bad])


def test_weights_offsets_past_32_bits():
    x = Held([90, 70], 2, 64, 64, 64, BF, seed=12)
    q = x.q(1, 4)
    lse = kv.kv4_decode(q, x.cache, x.t, x.l)[1]
    plain = kv.kv4_weights(q, x.cache, x.t, x.l, lse, torch.zeros(2, 2, 90, device="cuda"))
    far = 2 ** 30 + 1024
    buf = torch.empty(3 * far + 90, device="cuda")
    w = buf.as_strided((2, 2, 90), (2 * far, far, 1))
    w.zero_()
    assert torch.equal(kv.kv4_weights(q, x.cache, x.t, x.l, lse, w), plain)


def test_weights_captured_with_other_lengths():
    x = Held([500, 3, 64, 0], 2, 128, 128, 64, BF, seed=13)
    q = x.q(1, 8)
    lens, lse, w = x.l.clone(), torch.zeros(4, 8, 1, device="cuda"), torch.zeros(4, 2, 512, device="cuda")
    kv.kv4_weights(q, x.cache, x.t, lens, lse, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.kv4_weights(q, x.cache, x.t, lens, lse, w)
    for other in ([500, 3, 64, 0], [17, 0, 33, 0], [0, 0, 0, 0], [499, 2, 1, 0]):
        lens.copy_(i32(other))
        lse.copy_(kv.kv4_decode(q, x.cache, x.t, lens)[1])
        w.fill_(2.0)
        g.replay()
        assert torch.equal(w, kv.kv4_weights(q, x.cache, x.t, lens, lse, torch.full_like(w, 2.0)))


@pytest.mark.parametrize("lens", [[50, 0, 700, 3], [5] * 2000])
def test_weights_of_no_queries(lens):
    """Nothing is added; what is set is 0, up to each length."""
    x = Held(lens, 3, 64, 64, 64, BF, seed=14)
    q, lse = x.q(1, 6)[:, :0], torch.empty(len(lens), 6, 0, device="cuda")
    held = torch.rand(len(lens), 3, 750, generator=x.g).cuda() + 1
    status = zero()
    assert torch.equal(kv.kv4_weights(q, x.cache, x.t, x.l, lse, held.clone(), status=status), held)
    got = kv.kv4_weights(q, x.cache, x.t, x.l, lse, held.clone(), accumulate=False, status=status)
    attn.query_status(status)
    past = torch.arange(750, device="cuda") >= x.l[:, None, None]
    assert torch.equal(got, torch.where(past, held, 0.0))
    lens = [-1] + lens[1:]
    got = kv.kv4_weights(q, x.cache, x.t, i32(lens), lse, held.clone(), accumulate=False, status=status)
    assert torch.equal(got[0], held[0]) and (got[1, :, :lens[1]] == 0).all()
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)


# ------------------------------------------------------------------ eviction

class Full:
    """A cache of random bytes whose sequences have these lengths."""

    def __init__(self, lens, h, dqk, dv, page, seed, cols=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.h, self.g = list(lens), page, h, g
        need = [-(-n // page) for n in lens]
        cols = cols or max(1, max(need, default=0)) + 1
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g).tolist()
        self.table, at = [], 0
        for n in need:
            self.table.append(perm[at:at + n] + [(-5, 10 ** 9)[i % 2] for i in range(cols - n)])
            at += n
        u8 = lambda d: torch.randint(0, 256, (pages, h, page, d), generator=g, dtype=torch.uint8)  # noqa: E731
        bf = lambda d: torch.randint(-2 ** 15, 2 ** 15, (pages, h, page, d), generator=g,  # noqa: E731
                                     dtype=torch.int16).view(BF)
        self.arrays = [u8(dqk // 2), bf(dqk // 32), u8(dv // 2), bf(dv // 32)]
        self.cache = kv.KV4Cache(*(a.cuda() for a in self.arrays))
        self.t = i32(self.table) if len(lens) else torch.empty(0, cols, dtype=torch.int32, device="cuda")
        self.l = i32(self.lens)
        self.cap = max(self.lens, default=0) + 3

    def weights(self, kind):
        shape = (len(self.lens), self.h, self.cap)
        if kind == "ties":  # few different ones
            return torch.randint(0, 4, shape, generator=self.g).float() / 8
        w = torch.exp(3 * torch.randn(shape, generator=self.g))
        if kind == "odd" and w.numel():
            flat = w.view(-1)
            for i, v in enumerate((0.0, -0.0, float("nan"), float("inf"), -float("inf"), -1.0, 1e-45, 3.4e38)):
                flat[torch.randint(0, flat.numel(), (flat.numel() // 20 + 1,), generator=self.g)] = v
        return w

    def same(self, arrays):
        c = self.cache
        for got, want in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), arrays):
            bits = torch.uint8 if want.dtype == torch.uint8 else torch.int16
            assert torch.equal(got.cpu().view(bits), want.view(bits))

    def check(self, keep, first=None, recent=0, kind="spread", inplace=True, head=None):
        w = self.weights(kind)
        want = [a.clone() for a in self.arrays]
        out = w.clone() if inplace else torch.full_like(w, 77.0)
        firsts = [0] * len(self.lens) if first is None else first
        seq, kept = boundedref.evict([a.view(torch.int16) if a.dtype == BF else a for a in want], self.table, self.lens,
                                     w, out, keep, firsts, recent)
        back = boundedref.pages_back(self.table, self.lens, keep, self.page)
        head = len(back) + 2 if head is None else head
        free, status, wd = torch.full((head + 3,), -9, dtype=torch.int32), zero(), w.cuda()
        freed, fh = free.cuda(), i32([head])
        od = wd if inplace else torch.full_like(wd, 77.0)
        r = kv.kv4_evict(self.cache, self.t, self.l, wd, keep=keep, first=None if first is None else i32(first),
                         recent=recent, weights_out=None if inplace else od, free_pages=freed, free_head=fh,
                         status=status)
        torch.cuda.synchronize()
        attn.query_status(status)
        assert r.seq_lens.tolist() == seq
        assert torch.equal(r.kept.cpu(), kept)
        assert r.weights is od and torch.equal(od.cpu().view(torch.int32), out.view(torch.int32))
        if not inplace:
            assert torch.equal(wd.cpu().view(torch.int32), w.view(torch.int32))
        self.same(want)
        assert r.free_head.tolist() == [head - len(back)] and fh.tolist() == [head]
        free[head - len(back):head] = torch.tensor(back, dtype=torch.int32)
        assert torch.equal(freed.cpu(), free)
        assert self.t.tolist() == self.table and self.l.tolist() == self.lens
        return r


SHORT = [0, 1, 2, 15, 16, 17, 40, 63, 64, 65, 66, 100, 129, 300, 511, 900]


@pytest.mark.parametrize("kind,inplace", [("spread", True), ("ties", False), ("odd", True)])
@pytest.mark.parametrize("dqk,dv,h,page", [(64, 64, 2, 16), (128, 128, 3, 64), (192, 128, 1, 32), (256, 256, 2, 128)])
@pytest.mark.parametrize("keep,first,recent", [(64, 0, 0), (1, 0, 0), (65, 4, 16), (300, 16, 400), (33, 40, 5), (899, 3, 7)])
def test_evict(keep, first, recent, dqk, dv, h, page, kind, inplace):
    x = Full(SHORT, h, dqk, dv, page, seed=keep + dqk)
    x.check(keep, [first] * len(SHORT), recent, kind, inplace)


def test_evict_first_tokens_of_each_sequence():
    x = Full([200, 200, 200, 200, 30, 200], 2, 128, 128, 32, seed=1)
    x.check(100, [0, 50, 100, 101, 2 ** 31 - 1, -7], 10)
    x = Full([200, 77], 2, 128, 128, 32, seed=2)
    x.check(60, None, 2 ** 31 - 1)


def test_evict_all_alike_keeps_the_first():
    x = Full([333], 2, 64, 64, 64, seed=3)
    w = torch.full((1, 2, 333), 0.25, device="cuda")
    r = kv.kv4_evict(x.cache, x.t, x.l, w, keep=100, first=i32([10]), recent=20)
    assert r.kept[0, 1].tolist() == list(range(80)) + list(range(313, 333))
    assert r.free_head is None


@pytest.mark.parametrize("lens,h,keep", [([200000], 1, 5000), ([140001, 3], 1, 139990), ([40000, 20000, 9], 2, 2048),
                                         ([70 + i % 60 for i in range(700)], 2, 64), ([3000] * 20, 8, 2999)])
def test_evict_batches(lens, h, keep):
    """More candidates than a cluster's shared memory holds, and more sequences than
    clusters run at a time."""
    x = Full(lens, h, 64, 64, 64, seed=len(lens) + keep)
    x.check(keep, [4] * len(lens), min(50, keep // 3), "spread")


@pytest.mark.parametrize("kind", ["ties", "odd"])
@pytest.mark.parametrize("lens,h,keep", [([100001, 90000, 66000], 2, 30000), ([9001] * 310, 1, 4000)])
def test_evict_long_with_equal_weights(lens, h, keep, kind):
    """Equal weights on the border, of candidates that shared memory does not hold: of a
    cluster of 8 blocks, of single ones."""
    x = Full(lens, h, 64, 64, 128, seed=keep)
    x.check(keep, [i % 7 for i in range(len(lens))], 100, kind)


def test_evict_again_and_again():
    """The budget of a running sequence: what stays is what a list says."""
    x = Full([257], 2, 128, 128, 16, seed=4)
    lens, w = [257], x.weights("spread")
    d = w.cuda()
    for keep in (200, 199, 100, 3, 1):
        want = [a.clone() for a in (t.cpu() for t in (x.cache.k_codes, x.cache.k_scales, x.cache.v_codes,
                                                      x.cache.v_scales))]
        out = w.clone()
        seq, kept = boundedref.evict([a.view(torch.int16) if a.dtype == BF else a for a in want], x.table, lens, w, out,
                                     keep, [1], 1)
        r = kv.kv4_evict(x.cache, x.t, i32(lens), d, keep=keep, first=i32([1]), recent=1)
        x.same(want)
        assert torch.equal(r.kept.cpu(), kept) and torch.equal(d.cpu(), out) and r.seq_lens.tolist() == seq
        lens, w = seq, out


def test_evict_lengths_and_pages_out_of_range():
    for bad in (-1, 113, 2 ** 31 - 1):
        x = Full([100, 50, 64], 2, 64, 64, 16, seed=5)
        x.lens[1] = 0
        x.cap = 112
        w, status = torch.rand(3, 2, 112).cuda(), zero()
        r = kv.kv4_evict(x.cache, x.t, i32([100, bad, 64]), w, keep=40, status=status)
        assert r.seq_lens.tolist() == [40, 0, 40] and (r.kept[1] == -1).all()
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
    # a page of one sequence outside the cache: the others are evicted, its other rows too
    x = Full([100, 100], 1, 64, 64, 16, seed=6)
    w = torch.arange(100.0).flip(0).expand(2, 1, 100).contiguous()  # the first stay
    w[:, :, 20:40] = 0.0
    for col in (1, 3):
        t, status = x.t.clone(), zero()
        t[0, col] = (-1, x.cache.num_pages)[col == 3]
        before = [a.clone() for a in (x.cache.k_codes, x.cache.v_codes)]
        kv.kv4_evict(x.cache, t, x.l, w.cuda(), keep=60, status=status)
        torch.cuda.synchronize()
        hole = set(range(x.cache.num_pages)) - {p for r in t.tolist() for p in r}
        for p in hole:
            assert torch.equal(before[0][p], x.cache.k_codes[p]) and torch.equal(before[1][p], x.cache.v_codes[p])
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)


def test_evict_free_list_without_room():
    x = Full([100, 100], 1, 64, 64, 16, seed=7)
    w = torch.rand(2, 1, 103).cuda()
    for head, n in ((9, 20), (21, 20), (-1, 20), (10, 9)):  # 10 pages would go back
        free, status = torch.full((n,), -9, dtype=torch.int32, device="cuda"), zero()
        r = kv.kv4_evict(x.cache, x.t, x.l, w.clone(), keep=20, free_pages=free, free_head=i32([head]), status=status)
        assert r.free_head.tolist() == [head] and (free == -9).all() and r.seq_lens.tolist() == [20, 20]
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
    free, status = torch.full((10,), -9, dtype=torch.int32, device="cuda"), zero()
    r = kv.kv4_evict(x.cache, x.t, x.l, w.clone(), keep=20, free_pages=free, free_head=i32([10]), status=status)
    assert r.free_head.tolist() == [0] and free.tolist() == x.table[0][2:7] + x.table[1][2:7]
    attn.query_status(status)


def test_evict_given_outputs_strides_and_other_stream():
    x = Full([150, 90, 40], 2, 128, 128, 32, seed=8)
    buf = torch.rand(2, 3, 200).cuda()
    w = buf.transpose(0, 1)[..., 5:158]
    want, keep = w.cpu().clone(), buf.cpu().clone()
    arrays = [a.clone() for a in x.arrays]
    seq, kept = boundedref.evict([a.view(torch.int16) if a.dtype == BF else a for a in arrays], x.table, x.lens,
                                 w.cpu().clone(), want, 64, [0] * 3, 8)
    out = dict(kept=torch.zeros(3, 2, 64, dtype=torch.int32, device="cuda"),
               seq_lens_out=torch.zeros(3, dtype=torch.int32, device="cuda"))
    wide = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + x.t.shape[1]] = x.t
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    r = kv.kv4_evict(x.cache, wide[:, 3:3 + x.t.shape[1]], x.l, w, keep=64, recent=8, stream=s, **out)
    s.synchronize()
    assert r.kept is out["kept"] and r.seq_lens is out["seq_lens_out"] and r.seq_lens.tolist() == seq
    assert torch.equal(r.kept.cpu(), kept) and torch.equal(w.cpu(), want)
    x.same(arrays)
    assert torch.equal(buf.cpu()[..., :5], keep[..., :5]) and torch.equal(buf.cpu()[..., 158:], keep[..., 158:])


def test_evict_captured_with_other_lengths():
    x = Full([500, 300, 64], 2, 128, 128, 64, seed=9)
    lens, w0 = x.l.clone(), torch.rand(3, 2, 512)
    w = w0.cuda()
    arrays = lambda: (x.cache.k_codes, x.cache.k_scales, x.cache.v_codes, x.cache.v_scales)  # noqa: E731
    out = dict(kept=torch.zeros(3, 2, 100, dtype=torch.int32, device="cuda"),
               seq_lens_out=torch.zeros(3, dtype=torch.int32, device="cuda"))
    g = torch.cuda.CUDAGraph()
    kv.kv4_evict(x.cache, x.t, lens, w, keep=100, recent=3, **out)
    with torch.cuda.graph(g):
        kv.kv4_evict(x.cache, x.t, lens, w, keep=100, recent=3, **out)
    for other in ([500, 300, 64], [101, 100, 0], [77, 299, 64]):
        for a, b in zip(arrays(), x.arrays):
            a.copy_(b)
        w.copy_(w0)
        lens.copy_(i32(other))
        g.replay()
        want, wo = [a.clone() for a in x.arrays], w0.clone()
        seq, kept = boundedref.evict([a.view(torch.int16) if a.dtype == BF else a for a in want], x.table, other, w0,
                                     wo, 100, [0] * 3, 3)
        x.same(want)
        assert torch.equal(out["kept"].cpu(), kept) and out["seq_lens_out"].tolist() == seq
        assert torch.equal(w.cpu(), wo)


def test_evict_nothing():
    x = Full([], 2, 64, 64, 16, seed=10)
    r = kv.kv4_evict(x.cache, x.t, x.l, torch.empty(0, 2, 5, device="cuda"), keep=3, free_pages=i32([4, 5]),
                     free_head=i32([1]))
    assert r.free_head.tolist() == [1] and r.kept.shape == (0, 2, 3)


def test_evict_a_shared_prefix_stays_in_place():
    """Two sequences whose first pages are the same ones: `first` covers them, so no row
    of theirs is written."""
    x = Full([200, 200], 2, 128, 128, 32, seed=11)
    x.table[1][:3] = x.table[0][:3]
    x.t.copy_(i32(x.table))
    x.check(150, [96, 96], 10)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("keep", [1, 40, 64, 127, 128, 129])
def test_evict_gives_no_page_of_protected_tokens_back(page, keep):
    """Sequences over one prefix of 128 tokens, longer than the budget or not: its pages stay
    out of the free list, the sequences' own ones come back once each."""
    x = Full([200, 131, 128, 300, 250], 2, 64, 64, page, seed=12)
    for row in x.table[1:4]:
        row[:128 // page] = x.table[0][:128 // page]
    x.t.copy_(i32(x.table))
    first = [128, 128, 128, 128, 2 ** 31 - 1]  # (the last one is protected as a whole)
    back = [x.table[b][j] for b, n in enumerate(x.lens) if n > keep
            for j in range(-(-max(keep, min(first[b], n)) // page), -(-n // page))]
    assert len(set(back)) == len(back) > 0
    # what no longer fits the list, and what does
    for head in (len(back) - 1, len(back)):
        free, status = torch.full((40,), -9, dtype=torch.int32, device="cuda"), zero()
        before = [a.clone() for a in (x.cache.k_codes, x.cache.v_codes)] if keep <= 128 else []
        r = kv.kv4_evict(x.cache, x.t, x.l, x.weights("spread").cuda(), keep=keep, first=i32(first), free_pages=free,
                         free_head=i32([head]), status=status)
        assert r.seq_lens.tolist() == [min(n, keep) for n in x.lens]
        if head < len(back):
            assert r.free_head.tolist() == [head] and (free == -9).all()
            with pytest.raises(attn.AttnError, match="out of range"):
                attn.query_status(status)
        else:
            assert r.free_head.tolist() == [0] and free.tolist() == back + [-9] * (40 - len(back))
            attn.query_status(status)
        for a, b in zip(before, (x.cache.k_codes, x.cache.v_codes)):
            assert torch.equal(a, b)  # (nothing to move: what stays is the first tokens)
        stay = torch.arange(keep, dtype=torch.int32)
        for b, n in enumerate(x.lens):
            if n > keep and keep <= 128:
                assert torch.equal(r.kept[b].cpu(), stay.expand(2, -1))


def test_evict_largest_batch_with_a_free_list():
    """Every sequence gives a page back."""
    b, page = 2 ** 16, 16
    c = kv.KV4Cache.empty(2 * b, 1, 64, 64, page_size=page)
    g = torch.Generator(device="cuda").manual_seed(13)
    table = torch.randperm(2 * b, generator=g, device="cuda").int().view(b, 2)
    free, status = torch.full((b + 5,), -9, dtype=torch.int32, device="cuda"), zero()
    lens, w = torch.full((b,), 17, dtype=torch.int32, device="cuda"), torch.zeros(b, 1, 17, device="cuda")
    r = kv.kv4_evict(c, table, lens, w, keep=16, free_pages=free, free_head=i32([b + 2]), status=status)
    attn.query_status(status)
    assert r.free_head.tolist() == [2] and torch.equal(free[2:b + 2], table[:, 1])
    assert (free[:2] == -9).all() and (free[b + 2:] == -9).all() and (r.seq_lens == 16).all()


@pytest.mark.parametrize("page_id", [-1, -2 ** 31, 10 ** 9, None])
@pytest.mark.parametrize("col", [0, 1, 2, 3, 5, 7])
def test_evict_around_a_page_outside_the_cache(col, page_id):
    """Rows that come from or go to such a page stay as they are, every other row of that
    sequence and of the others moves, weights and lists are as without it; if the page goes back it does as
    -1.  Only a page that nothing moves in and that does not go back is not noticed."""
    x = Full([128, 100, 70], 2, 128, 128, 16, seed=14)
    keep, first, recent = 60, [20, 20, 0], 7
    x.table[0][col] = x.cache.num_pages if page_id is None else page_id
    t, w = i32(x.table), x.weights("spread")
    want, out = [a.clone() for a in x.arrays], w.clone()
    kept = torch.full((3, 2, keep), -1, dtype=torch.int32)
    for b, n in enumerate(x.lens):
        for a in range(2):
            src = boundedref.stays(w[b, a, :n].tolist(), keep, first[b], recent)
            kept[b, a] = torch.tensor(src, dtype=torch.int32)
            out[b, a, :keep] = w[b, a, src]
            place = lambda j: (x.table[b][j // 16], j % 16)  # noqa: E731
            moves = [(place(j), place(i)) for i, j in enumerate(src)]
            for was, arr in zip(x.arrays, want):
                for (p0, r0), (p1, r1) in moves:
                    if 0 <= p0 < x.cache.num_pages and 0 <= p1 < x.cache.num_pages:
                        arr[p1, a, r1] = was[p0, a, r0]
    back = [p if 0 <= p < x.cache.num_pages else -1 for p in boundedref.pages_back(x.table, x.lens, keep, 16)]
    free, status, wd = torch.full((30,), -9, dtype=torch.int32, device="cuda"), zero(), w.cuda()
    r = kv.kv4_evict(x.cache, t, x.l, wd, keep=keep, first=i32(first), recent=recent, free_pages=free,
                     free_head=i32([25]), status=status)
    torch.cuda.synchronize()
    x.same(want)
    assert torch.equal(r.kept.cpu(), kept) and torch.equal(wd.cpu(), out) and r.seq_lens.tolist() == [keep] * 3
    assert r.free_head.tolist() == [25 - len(back)] and free.tolist() == [-9] * (25 - len(back)) + back + [-9] * 5
    assert (-1 in back) == (col >= 4)
    if col == 0:
        attn.query_status(status)
    else:
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_weights_beside_an_infinite_scale(sign):
    """It changes its own token's entry of its head alone."""
    x = Held([200, 200], 2, 128, 128, 64, BF, seed=15)
    q = x.q(1, 8)
    lse = kv.kv4_decode(q, x.cache, x.t, x.l)[1]
    w = kv.kv4_weights(q, x.cache, x.t, x.l, lse, torch.ones(2, 2, 200, device="cuda"))
    x.cache.k_scales[x.table[0][1], 1, 7, 2] = sign * float("inf")
    got = kv.kv4_weights(q, x.cache, x.t, x.l, lse, torch.ones(2, 2, 200, device="cuda"))
    other = torch.ones_like(w, dtype=torch.bool)
    other[0, 1, 71] = False
    assert torch.equal(got[other], w[other])
