"""Attention over the cache for batches that share prefixes, on the GPU, against the
float64 form in kvref.py and against attn_kv_decode.

Bounds as in test_gpu_kv.py (u: half a step of the output's type, probabilities 2^-11):
the shared part's scores come from products that are exact up to elements 2^-37 of a
tile's largest, its probabilities are rounded once, and the parts are joined in FP32."""
import math

import pytest
import torch

import kvref
from bwd_tcgen05_tmem_gb300 import attn, kv
from test_gpu_kv import BF, FP, UNIT, empty_cache, i32

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


class Groups:
    """Requests of groups [(shared tokens, [own tokens of each member])] in a cache whose
    other bytes are poison.  Whole pages of a prefix are held once."""

    def __init__(self, groups, h, dqk, dv, page, dt, seed, vscale=1.0, loose=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.dt, self.g = page, dt, g
        self.starts, self.shared, self.lens, rows = [loose], [], [40] * loose, [(0, 40, None)] * loose
        for n, own in groups:
            n = n // page * page  # what lies in whole pages
            self.shared.append(n)
            for i, m in enumerate(own):
                self.lens.append(n + m)
                rows.append((n, m, len(self.shared) - 1))
            self.starts.append(len(self.lens))
        cols = max([1] + [-(-n // page) for n in self.lens]) + 1
        need = sum(n // page for n in self.shared) + sum(-(-m // page) for _, m, _ in rows)
        perm = torch.randperm(need + 2, generator=g).tolist()
        heads, at = [], 0
        for n in self.shared:
            heads.append(perm[at:at + n // page])
            at += n // page
        self.table = []
        for n, m, grp in rows:
            k = -(-m // page)
            row = (heads[grp] if grp is not None else []) + perm[at:at + k]
            at += k
            self.table.append(row + [(-5, 10 ** 9)[i % 2] for i in range(cols - len(row))])
        self.cache = empty_cache(need + 2, h, dqk, dv, page)
        slots = sorted({self.table[b][j // page] * page + j % page for b, n in enumerate(self.lens) for j in range(n)})
        self.k = torch.randn(len(slots), h, dqk, generator=g).to(dt)
        self.v = (torch.randn(len(slots), h, dv, generator=g) * vscale).to(dt)
        self.slots = slots
        self.write()
        self.t, self.l, self.s, self.n = i32(self.table), i32(self.lens), i32(self.starts), i32(self.shared)

    def write(self):
        if self.slots:
            kv.kv4_write(self.cache, self.k.cuda(), self.v.cuda(), i32(self.slots))

    def q(self, sq, hq, scale=1.5):
        return (torch.randn(len(self.lens), sq, hq, self.cache.d_qk, generator=self.g) * scale).to(self.dt).cuda()

    def reference(self, q, **kw):
        c = self.cache
        kc, vc = kvref.unpack(c.k_codes, True).cuda(), kvref.unpack(c.v_codes, False).cuda()
        safe = [[p if 0 <= p < c.num_pages else 0 for p in r] for r in self.table]
        return kvref.decode(q.double(), kc, c.k_scales.double(), vc, c.v_scales.double(), safe, self.lens,
                            kw.pop("scale", 1 / math.sqrt(c.d_qk)), **kw)

    def call(self, q, **kw):
        return kv.kv4_decode_shared(q, self.cache, self.t, self.l, self.s, self.n, **kw)

    def check(self, q, **kw):
        status = zero()
        o, lse = self.call(q, status=status, **kw)
        o2, lse2 = self.call(q, **kw)
        attn.query_status(status)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        within(o, lse, self.reference(q, scale=kw.get("scale", 1 / math.sqrt(self.cache.d_qk))))
        return o, lse


def within(o, lse, ref):
    """Probabilities of 11 bits, one rounding of the output; scores and sums as in
    test_gpu_kv.within."""
    ro, rl, mag, big = ref
    out = UNIT[o.dtype] if o.dtype != torch.float32 else 2.0 ** -24
    assert torch.isfinite(o).all()
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o[empty.transpose(1, 2)] == 0).all()
    score = 2.0 ** -20 * big
    err = (lse.double() - rl)[~empty].abs()
    assert (err <= score[~empty] + 2.0 ** -21 * rl[~empty].abs() + 2.0 ** -19).all(), float(err.max())
    tol = out * ro.abs() + (2.0 ** -11 + 2.0 ** -13) * mag + score.transpose(1, 2)[..., None] * mag + 2.0 ** -25
    err = (o.double() - ro).abs()
    assert (err <= tol).all(), (float((err - tol).max()), float((err / tol).max()))


DIMS = [(64, 64), (128, 128), (192, 128), (256, 256)]


def test_shared_smallest():
    """One tile of keys, two requests."""
    x = Groups([(128, [1, 1])], 1, 128, 128, 64, BF, seed=1)
    x.check(x.q(1, 4))


@pytest.mark.parametrize("dqk,dv", DIMS)
def test_shared_two_row_tiles(dqk, dv):
    x = Groups([(256, [3] * 70)], 1, dqk, dv, 64, BF, seed=2)
    x.check(x.q(1, 4))


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("dqk,dv", DIMS)
@pytest.mark.parametrize("hkv,group,sq,page", [(2, 4, 1, 64), (1, 1, 3, 16), (2, 8, 2, 32), (3, 5, 1, 128),
                                               (1, 12, 5, 256)])
def test_shared(dqk, dv, hkv, group, sq, page, dt):
    x = Groups([(300, [5, 64, 100, 7]), (1200, [70, 5]), (64, [5, 9, 11]), (30, [40, 50]), (700, [33, 300, 5, 6, 7])],
               hkv, dqk, dv, page, dt, seed=dqk + group, loose=2)
    x.check(x.q(sq, hkv * group))


@pytest.mark.parametrize("dqk,dv", DIMS)
@pytest.mark.parametrize("members,group,sq", [(2, 1, 1), (32, 4, 1), (33, 4, 1), (64, 4, 1), (65, 4, 1), (100, 8, 1),
                                              (7, 5, 9), (3, 16, 30)])
def test_shared_row_counts(members, group, sq, dqk, dv):
    x = Groups([(448, [sq + i % 5 for i in range(members)])], 2, dqk, dv, 64, BF, seed=members)
    x.check(x.q(sq, 2 * group))


@pytest.mark.parametrize("tokens", [64, 128, 192, 256, 320, 4096, 20000])
@pytest.mark.parametrize("dqk,dv", DIMS)
def test_shared_lengths(tokens, dqk, dv):
    x = Groups([(tokens, [1, 2, 3, 64, 65])], 2, dqk, dv, 32, FP, seed=tokens)
    x.check(x.q(1, 8))


def test_shared_many_groups():
    """More groups than threads of the first kernel, most of one request, and empty ones."""
    groups = [(64 * (i % 4), [1 + i % 3] * (1 + i % 3)) for i in range(1500)]
    x = Groups(groups, 1, 64, 64, 64, BF, seed=3)
    x.check(x.q(1, 2))


@pytest.mark.parametrize("vscale", [1e-4, 1e-2, 1000.0])
def test_shared_small_and_large_values(vscale):
    x = Groups([(700, [40, 1, 2])], 2, 128, 128, 64, FP, seed=4, vscale=vscale)
    x.check(x.q(1, 8))
    x.check(x.q(1, 8, scale=20.0))  # a sharp softmax


@pytest.mark.parametrize("dqk,dv", [(128, 128), (256, 256)])
@pytest.mark.parametrize("step", [2.0, 2.0 ** 5, 2.0 ** 19])
def test_shared_values_that_grow(step, dqk, dv):
    """Tiles whose V (and K) scales grow or shrink by a factor, so that O's unit moves;
    each row's values count by their own size (bf16 holds them)."""
    x = Groups([(1024, [3] * 40)], 1, dqk, dv, 64, BF, seed=5)
    at = torch.arange(len(x.slots))
    for power in (at // 128 % 5, 4 - at // 128 % 5):
        f = (step ** power.double())[:, None, None]
        x.v = (torch.randn(x.v.shape, generator=x.g).double() * f).to(BF)
        x.k = (torch.randn(x.k.shape, generator=x.g).double() * torch.where(f > 1, 0.5, 1.0)).to(BF)
        x.write()
        x.check(x.q(1, 4))


def test_shared_values_of_nothing():
    """Quarters of tiles whose V is zero, or 2^-60 of the others, still count in the sum."""
    x = Groups([(1024, [3] * 40)], 1, 128, 128, 64, BF, seed=16)
    at = torch.arange(len(x.slots)) // 32 % 4
    for small in (0.0, 2.0 ** -60, 2.0 ** -100):
        x.v = (torch.randn(x.v.shape, generator=x.g) * torch.where(at == 1, small, 1.0)[:, None, None]).to(BF)
        x.write()
        x.check(x.q(1, 4))


def test_shared_scores_far_apart():
    """Rows whose maximum moves by hundreds from tile to tile, and back."""
    x = Groups([(1024, [3] * 40)], 1, 128, 128, 64, BF, seed=6)
    x.k[:, :, 0] = (torch.arange(len(x.slots)) // 100 % 7 * 60.0 - 100.0)[:, None].to(BF)
    x.write()
    x.check(x.q(1, 4, scale=3.0))


def test_shared_scale_output_type_and_given_buffers():
    x = Groups([(320, [9, 33, 2])], 2, 128, 128, 32, BF, seed=7)
    q = x.q(2, 6)
    x.check(q, scale=0.3)
    o, lse = x.check(q, o_dtype=torch.float32)
    out = torch.full((3, 6, 2, 136), 7.0, dtype=BF, device="cuda").transpose(1, 2)[..., :128]
    ws = torch.full((kv.decode_shared_workspace_size(q, x.cache, x.t, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(3, 10, 2, 128, dtype=BF, device="cuda")
    wide[:, 2:8] = q.transpose(1, 2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, lse2 = x.call(wide[:, 2:8].transpose(1, 2), out=out, workspace=ws, stream=s)
    s.synchronize()
    assert o2 is out and torch.equal(lse2, lse)
    assert torch.equal(o2, o.to(BF))


def test_shared_agrees_with_decode():
    """The same requests with and without the promise: within twice the bound of either."""
    x = Groups([(2048, [17] * 20), (512, [4] * 3)], 2, 128, 128, 64, BF, seed=8)
    q = x.q(1, 8)
    a, la = x.call(q, o_dtype=torch.float32)
    b, lb = kv.kv4_decode(q, x.cache, x.t, x.l, o_dtype=torch.float32)
    mag = x.reference(q)[2]
    assert ((a - b).abs() <= 2.0 ** -10 * mag + 2.0 ** -16 * mag + 2.0 ** -24).all()
    assert (la - lb).abs().max() <= 2.0 ** -15


def test_shared_requests_that_do_not_fit():
    """Idle requests, ones shorter than the prefix, and one with as many tokens as it has
    (and the newest): each reads its own row of the table."""
    x = Groups([(640, [1, 5, 7, 20, 3, 2])], 2, 128, 128, 64, BF, seed=9)
    for change in ({0: 0}, {0: 0, 1: 0, 2: 0}, {1: 640, 3: 641}, {0: 100, 5: 639}, {i: 0 for i in range(5)},
                   {i: 0 for i in range(6)}):
        for b, n in change.items():
            x.lens[b] = n
        x.l = i32(x.lens)
        for sq in (1, 3):
            x.check(x.q(sq, 8))


def test_shared_groups_and_lengths_out_of_range():
    x = Groups([(256, [5, 6]), (128, [7, 8, 9])], 1, 64, 64, 64, BF, seed=10)
    q = x.q(1, 4)
    ref = x.reference(q)
    cap = x.t.shape[1] * 64
    for starts, shared in (([0, 6, 5], x.shared), ([-1, 2, 5], x.shared), ([0, 3, 2], x.shared), ([0, 2, 2 ** 31 - 1], x.shared),
                           (x.starts, [-1, 128]), (x.starts, [cap + 1, 128]), (x.starts, [2 ** 31 - 1, -2 ** 31])):
        status = zero()
        o, lse = kv.kv4_decode_shared(q, x.cache, x.t, x.l, i32(starts), i32(shared), status=status)
        within(o, lse, ref)  # what is left is not shared
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
    for bad in (-1, cap + 1, 2 ** 31 - 1):
        status, lens = zero(), list(x.lens)
        lens[3] = bad
        o, lse = kv.kv4_decode_shared(q, x.cache, x.t, i32(lens), x.s, x.n, status=status)
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
        assert (o[3] == 0).all() and torch.isneginf(lse[3]).all()
        keep = [0, 1, 2, 4]
        within(o[keep], lse[keep], [r[keep] for r in ref])
    # a page outside the cache: the other group is right
    t = x.t.clone()
    t[:2, 1] = x.cache.num_pages
    status = zero()
    o, lse = kv.kv4_decode_shared(q, x.cache, t, x.l, x.s, x.n, status=status)
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)
    within(o[2:], lse[2:], [r[2:] for r in ref])


def test_shared_prefix_longer_than_promised_pages():
    """A shorter promise, down to none, gives the same within the bounds."""
    x = Groups([(700, [20, 30, 40])], 1, 128, 128, 16, BF, seed=11)
    q = x.q(1, 4)
    ref = x.reference(q)
    for n in (0, 1, 63, 64, 65, 127, 129, 400, 688):
        o, lse = kv.kv4_decode_shared(q, x.cache, x.t, x.l, x.s, i32([n]))
        within(o, lse, ref)


def test_shared_nan_and_infinity():
    x = Groups([(256, [5, 6, 7]), (256, [5, 6])], 2, 128, 128, 64, BF, seed=12)
    q = x.q(1, 8)
    good = x.call(q)
    page = x.table[0][1]
    # a NaN in V reaches the dims of its group, of one kv head and the group's requests
    x.cache.v_scales[page, 1, 9, 2] = float("nan")
    o, lse = x.call(q)
    bad = torch.isnan(o)
    assert bad[:3, :, 4:, 64:96].all() and int(bad.sum()) == 3 * 4 * 32
    assert torch.equal(o[~bad], good[0][~bad]) and torch.equal(lse, good[1])
    # one in K all of those requests' rows of that head
    x.cache.k_scales[page, 0, 9, 2] = float("nan")
    o, lse = x.call(q)
    assert torch.isnan(lse[:3, :4]).all() and torch.isnan(o[:3, :, :4]).all()
    assert torch.equal(lse[3:], good[1][3:]) and torch.equal(o[3:], good[0][3:])
    assert torch.equal(lse[:3, 4:], good[1][:3, 4:])


def test_shared_captured_with_other_lengths():
    x = Groups([(640, [9, 70, 20]), (128, [3, 4])], 2, 128, 128, 64, BF, seed=13)
    q = x.q(1, 8)
    lens, starts, shared = x.l.clone(), x.s.clone(), x.n.clone()
    ws = torch.empty(kv.decode_shared_workspace_size(q, x.cache, x.t, 2), dtype=torch.uint8, device="cuda")
    o, lse = kv.kv4_decode_shared(q, x.cache, x.t, lens, starts, shared, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.kv4_decode_shared(q, x.cache, x.t, lens, starts, shared, workspace=ws, out=o, lse=lse)
    for a, b, c in ((x.lens, x.starts, x.shared), ([649, 0, 641, 130, 131], [0, 3, 5], [640, 64]),
                    ([649, 700, 641, 130, 131], [0, 3, 3], [128, 0]), ([0] * 5, [0, 3, 5], [640, 128])):
        lens.copy_(i32(a))
        starts.copy_(i32(b))
        shared.copy_(i32(c))
        ws.fill_(0xFF)
        g.replay()
        want = kv.kv4_decode_shared(q, x.cache, x.t, lens, starts, shared)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_shared_two_streams_at_once():
    x = Groups([(4096, [9] * 40)], 2, 128, 128, 64, BF, seed=14)
    q = [x.q(1, 8) for _ in range(2)]
    want = [x.call(a) for a in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(kv.decode_shared_workspace_size(q[0], x.cache, x.t, 1), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    outs = [(torch.empty_like(want[0][0]), torch.empty_like(want[0][1])) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            x.call(q[i], workspace=ws[i], out=outs[i][0], lse=outs[i][1], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def test_shared_nothing():
    x = Groups([(64, [1, 2])], 1, 64, 64, 64, BF, seed=15)
    q = x.q(1, 2)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    o, lse = kv.kv4_decode_shared(q, x.cache, x.t, x.l, i32([0]), none)
    a, b = kv.kv4_decode(q, x.cache, x.t, x.l)
    assert torch.equal(o, a) and torch.equal(lse, b)
    o, lse = kv.kv4_decode_shared(q[:0], x.cache, x.t[:0], x.l[:0], i32([0]), none)
    assert o.shape == (0, 1, 2, 64)


@pytest.mark.parametrize("dropped", [0, 1, 5])
@pytest.mark.parametrize("members", [3, 40])
@pytest.mark.parametrize("dqk,dv", DIMS)
def test_shared_wait_that_runs_out(dqk, dv, members, dropped):
    """One tile's K is never announced, and the first block gives up after 20 ms: the call
    returns, says so, and its rows (of the first kv head's first row tile) are NaN instead of
    numbers that take an earlier call's parts; the others and the next call are right.
    (3 requests: the softmax groups take turns; 40: they have rows of their own.)"""
    x = Groups([(40960, [3] * members), (128, [5, 6])], 2, dqk, dv, 64, BF, seed=17, loose=2)
    q, status = x.q(1, 8), zero()
    ws = torch.empty(kv.decode_shared_workspace_size(q, x.cache, x.t, 2), dtype=torch.uint8, device="cuda")
    o, lse = x.call(q, workspace=ws, status=status)
    attn.query_status(status)
    for word in (status, None):
        attn.debug_inject(attn.DEBUG_SHARED, dropped, 20_000_000)
        bad, bad_lse = x.call(q, workspace=ws, status=word)
        lost = torch.zeros(len(x.lens), 8, dtype=torch.bool, device="cuda")
        lost[2:2 + min(members, 32 if dv > 128 else 64), :4] = True  # 128 or 256 rows, 4 of a request
        assert torch.equal(torch.isnan(bad_lse[:, :, 0]), lost) and torch.equal(bad_lse[:, :, 0][~lost], lse[:, :, 0][~lost])
        assert torch.isnan(bad[:, 0][lost]).all() and torch.equal(bad[:, 0][~lost], o[:, 0][~lost])
    with pytest.raises(attn.AttnError) as e:
        attn.query_status(status)
    assert e.value.code == 6  # ATTN_ERR_TIMEOUT
    status.zero_()
    o2, lse2 = x.call(q, workspace=ws, status=status)
    attn.query_status(status)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("sq", [1, 3])
@pytest.mark.parametrize("bad", [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 2, -2 ** 31 + 3, -300])
def test_shared_lengths_far_below_zero(bad, sq):
    """They count as 0 too, so their requests share nothing (and leave a group of two alone)."""
    x = Groups([(256, [5, 6, 7]), (192, [8, 9])], 1, 64, 64, 64, BF, seed=18)
    q = x.q(sq, 4)
    ref = x.reference(q)
    for at in (1, 4):
        status, lens = zero(), list(x.lens)
        lens[at] = bad
        o, lse = kv.kv4_decode_shared(q, x.cache, x.t, i32(lens), x.s, x.n, status=status)
        with pytest.raises(attn.AttnError, match="out of range"):
            attn.query_status(status)
        assert (o[at] == 0).all() and torch.isneginf(lse[at]).all()
        keep = [b for b in range(5) if b != at]
        within(o[keep], lse[keep], [r[keep] for r in ref])


@pytest.mark.parametrize("hidden", [-80, -18])
@pytest.mark.parametrize("large", [0, 12, 16, 20, 24, 28])
@pytest.mark.parametrize("where", ["first", "last"])
def test_shared_many_small_probabilities_beside_large_values(large, where, hidden):
    """One token of probability 0.6 and 960 that share the rest, beside a tile of V scales 2^k
    times theirs that nobody looks at, or hardly: a token's probability p enters as p 2^(11 + e - r), 2^e its V
    scale's exponent and 2^r the reference, at most twice the largest product m of a probability and a
    V scale; half a step below fp16's normal range, 2^-25, is 2^(-36 - e + r) |v| in O, |v| < 2^(e + 4): 2^-31 m.
    (As many heads as blocks, so that a block's run holds the whole prefix, and all of it in even
    tiles: the softmax groups take turns.)"""
    h, n, dt = 160, 1024, BF
    x = Groups([(n, [1, 1])], h, 64, 64, 64, dt, seed=19)
    scale, q0 = 1 / 8, 8.0
    of = lambda p: math.log(p) / (scale * q0)  # noqa: E731  (dim 0 of a key whose probability is p times the largest's)
    slots = {s: i for i, s in enumerate(x.slots)}
    at = torch.tensor([slots[x.table[0][j // 64] * 64 + j % 64] for j in range(n)])
    big = at[:64] if where == "first" else at[-128:-64]
    x.k.zero_()
    x.v.fill_(1.0)
    x.k[:, :, 0] = of(1.37 * 2.0 ** -11)
    x.k[at[520], :, 0] = 0.0
    x.k[big, :, 0] = of(2.0 ** hidden)
    x.v[big] = 2.0 ** large
    x.write()
    q = torch.zeros(2, 1, h, 64)
    q[..., 0] = q0
    q = q.to(dt).cuda()
    status = zero()
    o, lse = x.call(q, o_dtype=torch.float32, status=status)
    attn.query_status(status)
    ro, rl, mag, _ = x.reference(q)
    p_max = torch.exp(-rl).transpose(1, 2)[..., None]  # (the largest score is 0, scales are 1 / 7 and 2^large / 7)
    most = 1.01 / 7 * max(1.0, 2.0 ** (large + hidden + 0.2))  # (0.2: of K's scale in bf16, 2^-8 of 80 and less)
    err = (o.double() - ro).abs()
    assert (err <= (2.0 ** -11 + 2.0 ** -13) * mag + n * 2.0 ** -31 * most * p_max).all(), float(err.max())
    assert (lse.double() - rl).abs().max() <= 2.0 ** -19 + 2.0 ** -20 * 8


@pytest.mark.parametrize("apart", [8, 20, 26, 30])
def test_shared_keys_of_very_different_scales(apart):
    """Every other token's K is 2^apart times the others' and far below them in score: what the
    others lose is at most 2^-32 of its scale an element (half a step of the scale's operand, 2^-25 below
    fp16's normal range, times 8 for the code, and one for the product, all in units of 2^-11 of the scale)."""
    x = Groups([(512, [3] * 5)], 1, 128, 128, 64, BF, seed=20)
    slots = {s: i for i, s in enumerate(x.slots)}
    at = torch.tensor([slots[x.table[0][j // 64] * 64 + j % 64] for j in range(512)])
    x.k[:, :, :32] = 0.0
    x.k = (x.k.double() * 2.0 ** -apart).to(BF)
    x.k[at[::2]] = 0.0
    x.k[at[::2], :, 0] = -1.0
    x.write()
    q = x.q(1, 4).double() * 2.0 ** apart
    q[..., 0] = 2.0 ** (apart + 5)
    q[..., 1:32] = 0.0
    q = q.to(BF)
    status = zero()
    o, lse = x.call(q, o_dtype=torch.float32, status=status)
    attn.query_status(status)
    ro, rl, mag, _ = x.reference(q)
    scale = 1 / math.sqrt(128)
    # of the tokens that count: 2^-20 of sum |q k|, and the loss beside a scale of 1 / 7
    small = x.k.double().cuda().clone()
    small[at[::2]] = 0.0
    d = scale * (2.0 ** -20 * (q.double().abs()[:, 0] @ small[:, 0].abs().T).amax(-1)
                 + 2.0 ** -32 / 7 * 1.01 * q.double().abs()[:, 0].sum(-1))[..., None]
    assert float(rl.min()) + 2.0 ** (apart + 4) * scale > 0  # (the large ones' scores are that far below 0)
    grow = torch.expm1(d)
    assert ((lse.double() - rl).abs() <= grow + 2.0 ** -21 * rl.abs() + 2.0 ** -19).all()
    tol = (2.0 ** -11 + 2.0 ** -13 + 2 * grow[:, None]) * mag + 2.0 ** -25
    assert ((o.double() - ro).abs() <= tol).all()


@pytest.mark.parametrize("dqk,dv", DIMS)
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("members", [3, 40])
def test_shared_infinite_scales(side, members, dqk, dv):
    """An infinite scale does to its own dims (of V) or rows (of K) what infinities and 0 * inf do in
    the formula, and nothing to the others, whose precision it must not take."""
    x = Groups([(256, [5] * members), (256, [5, 6])], 2, dqk, dv, 64, BF, seed=21)
    getattr(x.cache, side + "_scales")[x.table[0][1], 1, 9, 1] = float("inf")
    q, status = x.q(1, 8), zero()
    o, lse = x.call(q, status=status)
    attn.query_status(status)
    ro, rl, mag, big = x.reference(q)
    for got, want in ((o, ro), (lse, rl)):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.isinf(got), torch.isinf(want)) and (got[torch.isinf(got)] == want[torch.isinf(got)]).all()
    bad = ~torch.isfinite(ro)
    assert int(bad.sum()) == members * 4 * (dv if side == "k" else 32)
    fine = torch.isfinite(rl)
    within(torch.where(bad, 0.0, o), torch.where(fine, lse, 0.0), (torch.where(bad, 0.0, ro), torch.where(fine, rl, 0.0),
                                                                   torch.where(bad, 0.0, mag), torch.where(fine, big, 0.0)))
