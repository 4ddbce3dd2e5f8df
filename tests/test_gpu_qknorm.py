"""attn.qk_norm_rope and its gradient on the GPU against the float64 form.

Tolerances, from the arithmetic.  One rounding to the type: u |z| (u = 2^-8 bf16,
2^-11 fp16, half a step), 2^-25 for fp16 values below its normal range.  FP32
inside: the norm's sum has at most 48 terms a lane and 5 exchanges, a product
chain of 3 and a turn of 3 operations follow, each at most 2^-24: under 64 *
2^-24 = 2^-18 of the turned pair's length.  The gradient has two such sums:
2^-17 of the sizes that cancel.  A sum over n rows adds at most n + 64 roundings."""
import pytest
import torch

import kvref
from bwd_tcgen05_tmem_gb300 import attn

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


def make(b, s, hq, hk, d, dt, seed, wdt=torch.float32, spread=True):
    """q, k as slices of one projection, weights, gradients, positions."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    x = r(b, s, hq + hk + 1, d)
    if spread:  # rows of very different sizes
        x = x * torch.exp2(torch.randint(-8, 9, (b, s, hq + hk + 1, 1), generator=g).float())
    qkv = x.to(dt).cuda()
    pos = torch.randint(0, 5000, (b, s), generator=g, dtype=torch.int32).cuda()
    return dict(q=qkv[:, :, :hq], k=qkv[:, :, hq:hq + hk], wq=(1 + 0.3 * r(d)).to(wdt).cuda(),
                wk=(1 + 0.3 * r(d)).to(wdt).cuda(), dqo=r(b, s, hq, d).to(dt).cuda(),
                dko=r(b, s, hk, d).to(dt).cuda(), pos=pos)


def close(got, want, tol):
    got = got.double()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - tol
    assert (over <= 0).all(), (float(over.max()), float(tol.flatten()[over.argmax()]))


def pair_length(y, rot, inter):
    """sqrt of both squares of the pair that each element is turned with."""
    one = torch.ones(y.shape[:-2] + (rot // 2,), dtype=torch.float64, device=y.device)
    sq = kvref.turn(y.pow(2), one * 0, one, inter)  # (a, b) -> (-b, a)
    return (y.pow(2) + torch.where(torch.arange(y.shape[-1], device=y.device) < rot, sq.abs(), 0 * sq)).sqrt()


def check(m, cos, sin, inter, norm=True, weights=True, eps=1e-6, positions=True, b3=False):
    dt, d = m["q"].dtype, m["q"].shape[-1]
    u = UNIT[dt]
    rot = 0 if cos is None else 2 * cos.shape[1]
    wq, wk = (m["wq"], m["wk"]) if weights else (None, None)
    pos = m["pos"] if positions else None
    ts = [m["q"], m["k"], m["dqo"], m["dko"]]
    if b3:  # packed tensors
        ts = [t[0] for t in ts]
        pos = pos[0]
    kw = dict(positions=pos, wq=wq, wk=wk, norm=norm, eps=eps, interleaved=inter)
    zq, zk = attn.qk_norm_rope(ts[0], ts[1], cos, sin, **kw)
    grads = attn.qk_norm_rope_bwd(ts[0], ts[1], cos, sin, ts[2], ts[3], **kw)
    again = attn.qk_norm_rope_bwd(ts[0], ts[1], cos, sin, ts[2], ts[3], **kw)
    torch.cuda.synchronize()
    for a, b in zip(grads, again):
        assert (a is None and b is None) or torch.equal(a, b)
    at = (m["pos"] if positions else torch.arange(m["q"].shape[1], device="cuda").expand(m["q"].shape[:2])).long()
    c, s = (cos[at].double(), sin[at].double()) if rot else (None, None)
    n_rows = m["q"].shape[0] * m["q"].shape[1]
    for x, w, z, dz, dx, dw in ((m["q"], wq, zq, m["dqo"], grads[0], grads[2]),
                                (m["k"], wk, zk, m["dko"], grads[1], grads[3])):
        z, dx = z.view(x.shape), dx.view(x.shape)
        x64 = x.double().requires_grad_()
        w64 = None if w is None else w.double().requires_grad_()
        want = kvref.norm_rope(x64, w64, c, s, norm, eps, inter)
        y = kvref.norm_rope(x64, w64, None, None, norm, eps, inter).detach()
        length = pair_length(y, rot, inter) if rot else y.abs()
        close(z, want.detach(), u * want.detach().abs() + 2.0 ** -18 * length + 2.0 ** -25)
        (want * dz.double()).sum().backward()
        # the sizes that cancel in dx = r (g - x r^2 mean(g x))
        gl = pair_length(dz.double(), rot, inter) if rot else dz.double().abs()
        gl = gl if w is None else gl * w.double().abs()
        r = 1 / torch.sqrt(x.double().pow(2).mean(-1, keepdim=True) + eps) if norm else torch.ones_like(x.double()[..., :1])
        size = r * (gl + (x.double().abs() * r * r * (gl * x.double().abs()).mean(-1, keepdim=True) if norm else 0))
        close(dx, x64.grad, u * x64.grad.abs() + 2.0 ** -17 * size + 2.0 ** -25)
        if w is not None:
            total = (gl / w.double().abs() * (x.double() * r).abs()).sum((0, 1, 2))
            close(dw, w64.grad, 2.0 ** -24 * (n_rows * x.shape[2] + 64) * total)
        else:
            assert dw is None


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 128, True),
                                         (128, 16, False), (192, 192, False), (192, 64, True), (192, 96, False),
                                         (256, 256, True), (256, 64, False), (512, 512, False), (512, 256, True)])
def test_dims(d, rot, inter, dt):
    cos, sin = attn.rope_tables(5000, rot)
    check(make(2, 37, 5, 2, d, dt, seed=d + rot), cos, sin, inter)


@pytest.mark.parametrize("b,s,hq,hk", [(1, 1, 1, 1), (1, 1, 32, 8), (3, 1, 7, 7), (1, 301, 17, 1), (5, 3, 128, 2)])
def test_sizes_and_heads(b, s, hq, hk):
    cos, sin = attn.rope_tables(5000, 128)
    check(make(b, s, hq, hk, 128, BF, seed=s + hq), cos, sin, False)


@pytest.mark.parametrize("kw", [dict(norm=False, weights=False), dict(weights=False), dict(eps=0.1),
                                dict(positions=False), dict(norm=False, weights=False, positions=False)])
def test_without_norm_weights_or_positions(kw):
    cos, sin = attn.rope_tables(5000, 128)
    check(make(2, 19, 4, 2, 128, FP, seed=9), cos, sin, False, **kw)


def test_norm_alone_and_16_bit_weights():
    check(make(2, 19, 4, 2, 256, BF, seed=10), None, None, False)
    cos, sin = attn.rope_tables(5000, 64)
    check(make(2, 19, 4, 2, 64, BF, seed=11, wdt=BF), cos, sin, True)
    check(make(1, 19, 4, 2, 192, FP, seed=12, wdt=FP), cos, sin, True)


def test_packed():
    cos, sin = attn.rope_tables(5000, 128)
    check(make(1, 77, 4, 2, 128, BF, seed=13), cos, sin, False, b3=True)


def test_queries_alone_and_in_place():
    m = make(2, 50, 6, 2, 128, BF, seed=14)
    cos, sin = attn.rope_tables(5000, 128)
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])
    zq, zk = attn.qk_norm_rope(m["q"], m["k"], cos, sin, **kw)
    only, none = attn.qk_norm_rope(m["q"], None, cos, sin, positions=m["pos"], wq=m["wq"])
    assert none is None and torch.equal(only, zq)
    full = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)
    part = attn.qk_norm_rope_bwd(m["q"], None, cos, sin, m["dqo"], None, positions=m["pos"], wq=m["wq"])
    assert torch.equal(full[0], part[0]) and part[1] is None and part[3] is None
    n = m["q"].shape[0] * m["q"].shape[1] * m["q"].shape[2]
    assert torch.allclose(full[2], part[2], rtol=0, atol=float(2.0 ** -23 * n * full[2].abs().max()))
    # the gradient over the incoming one, the forward over the projection
    dqo, dko = m["dqo"].clone(), m["dko"].clone()
    attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, dqo, dko, dq=dqo, dk=dko, **kw)
    assert torch.equal(dqo, full[0]) and torch.equal(dko, full[1])
    attn.qk_norm_rope(m["q"], m["k"], cos, sin, q_out=m["q"], k_out=m["k"], **kw)
    assert torch.equal(m["q"], zq) and torch.equal(m["k"], zk)


def test_padding_rows_stay_and_add_nothing():
    m = make(2, 40, 4, 2, 128, BF, seed=15)
    cos, sin = attn.rope_tables(5000, 128)
    pad = torch.zeros(2, 40, dtype=torch.bool)
    pad[0, 33:], pad[1, 5], pad[1, 12:20] = True, True, True
    m["pos"][pad.cuda()] = -1
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])
    held = [torch.full_like(t, 7.0) for t in (m["dqo"], m["dko"])]
    z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, q_out=held[0].clone(), k_out=held[1].clone(), **kw)
    g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], dq=held[0].clone(), dk=held[1].clone(), **kw)
    poison = {n: t.clone() for n, t in m.items()}
    for n in ("q", "k", "dqo", "dko"):
        poison[n][pad.cuda()] = float("nan")
    z2 = attn.qk_norm_rope(poison["q"], poison["k"], cos, sin, q_out=held[0].clone(), k_out=held[1].clone(), **kw)
    g2 = attn.qk_norm_rope_bwd(poison["q"], poison["k"], cos, sin, poison["dqo"], poison["dko"],
                               dq=held[0].clone(), dk=held[1].clone(), **kw)
    for a, b in zip((*z, *g), (*z2, *g2)):
        assert torch.equal(a, b)
    for t in (*z, g[0], g[1]):
        assert (t[pad.cuda()] == 7.0).all() and torch.isfinite(t).all()


def test_positions_outside_the_tables_give_nan_and_a_status():
    m = make(1, 9, 4, 2, 128, BF, seed=16)
    cos, sin = attn.rope_tables(5000, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(wq=m["wq"], wk=m["wk"], status=status)
    attn.qk_norm_rope(m["q"], m["k"], cos, sin, positions=m["pos"], **kw)
    attn.query_status(status)
    m["pos"][0, 4], m["pos"][0, 6] = 5000, 2 ** 31 - 1
    z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, positions=m["pos"], **kw)
    for t in z:
        assert torch.isnan(t[0, [4, 6]]).all() and torch.isfinite(t[0, [0, 1, 2, 3, 5, 7, 8]]).all()
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)


def test_offsets_past_32_bits_and_broadcast_input():
    """Tokens 2^28 elements apart, and one row broadcast to all heads."""
    d, far = 128, 1 << 28
    big = torch.zeros(9 * far + 4 * d, dtype=BF, device="cuda")
    q = big.as_strided((1, 10, 4, d), (0, far, d, 1))
    g = torch.Generator().manual_seed(17)
    x = torch.randn(1, 10, 4, d, generator=g).to(BF).cuda()
    q.copy_(x)
    cos, sin = attn.rope_tables(16, d)
    z, _ = attn.qk_norm_rope(q, None, cos, sin)
    w, _ = attn.qk_norm_rope(x, None, cos, sin)
    assert torch.equal(z, w)
    attn.qk_norm_rope(x, None, cos, sin, q_out=q)
    assert torch.equal(q, w)
    one = x[:, :, :1].expand(1, 10, 4, d)
    z, _ = attn.qk_norm_rope(one, None, cos, sin)
    assert torch.equal(z, w[:, :, :1].expand(1, 10, 4, d))


def test_captured_and_on_another_stream():
    m = make(2, 33, 8, 2, 128, BF, seed=18)
    cos, sin = attn.rope_tables(5000, 128)
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])

    def step():
        z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, **kw)
        return (*z, *attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    m["q"].mul_(2)
    m["dko"].neg_()
    m["pos"].add_(-1).clamp_(min=-1)
    graph.replay()
    torch.cuda.synchronize()
    live = (m["pos"] >= 0)
    want = step()
    for a, b in zip(got, want):
        assert torch.equal(a, b) if a.dim() == 1 else torch.equal(a[live], b[live])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, stream=side, **kw)
    g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], stream=side, **kw)
    side.synchronize()
    for a, b in zip((*z, *g), want):
        assert torch.equal(a, b) if a.dim() == 1 else torch.equal(a[live], b[live])


def test_no_rows():
    cos, sin = attn.rope_tables(16, 128)
    q = torch.empty(2, 0, 4, 128, dtype=BF, device="cuda")
    w = torch.ones(128, device="cuda")
    z = attn.qk_norm_rope(q, q, cos, sin, wq=w, wk=w)
    g = attn.qk_norm_rope_bwd(q, q, cos, sin, q, q, wq=w, wk=w)
    assert z[0].shape == q.shape and (g[2] == 0).all() and (g[3] == 0).all()
    with pytest.raises(ValueError, match="shape"):
        attn.qk_norm_rope(q, q[..., :64], cos, sin)


def test_with_attention_training():
    """norm + rotation, attention forward and backward, and their gradient,
    against float64 autograd of the whole.  Bound: the relative L2 bound 0.008 of
    the attention gradients, plus the roundings of q, k and of their gradients."""
    import math
    b, s, hq, hk, d = 1, 192, 4, 2, 128
    m = make(b, s, hq, hk, d, BF, seed=19, spread=False)
    g = torch.Generator().manual_seed(20)
    v, do = (torch.randn(b, s, h, d, generator=g).to(BF).cuda() for h in (hk, hq))
    cos, sin = attn.rope_tables(5000, d)
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])
    q, k = attn.qk_norm_rope(m["q"], m["k"], cos, sin, **kw)
    o, lse = attn.fwd(q, k, v)
    dq, dk, dv = attn.bwd(q, k, v, o, do, lse)
    got = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, dq, dk, **kw)
    torch.cuda.synchronize()
    x = [m[n].double().requires_grad_() for n in ("q", "k", "wq", "wk")]
    c, sn = cos[m["pos"].long()].double(), sin[m["pos"].long()].double()
    q64 = kvref.norm_rope(x[0], x[2], c, sn, True, 1e-6, False).transpose(1, 2)
    k64 = kvref.norm_rope(x[1], x[3], c, sn, True, 1e-6, False).transpose(1, 2).repeat_interleave(hq // hk, 1)
    sc = q64 @ k64.transpose(-1, -2) / math.sqrt(d)
    sc = sc.masked_fill(torch.ones(s, s, device="cuda").triu(1).bool(), -math.inf)
    o64 = (sc.softmax(-1) @ v.double().transpose(1, 2).repeat_interleave(hq // hk, 1)).transpose(1, 2)
    (o64 * do.double()).sum().backward()
    for t, w in ((o, o64.detach()), *zip(got, [y.grad for y in x])):
        rel = float((t.double() - w).norm() / w.norm())
        assert rel < 0.008 + 4 * 2.0 ** -8 / 3 ** 0.5, rel


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (3, 2), (4, 3)])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_few_heads(hq, hk, d):
    """Several tokens share a warp where a token's heads leave it lanes."""
    cos, sin = attn.rope_tables(5000, 64)
    for b, s in ((1, 1), (1, 7), (3, 43)):
        check(make(b, s, hq, hk, d, BF, seed=d + hq + s), cos, sin, False)


def test_few_heads_with_padding_between_tokens():
    m = make(3, 21, 2, 1, 64, BF, seed=21)
    cos, sin = attn.rope_tables(5000, 64)
    kw = dict(wq=m["wq"], wk=m["wk"])
    whole = attn.qk_norm_rope(m["q"], m["k"], cos, sin, positions=m["pos"], **kw)
    full = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], positions=m["pos"], **kw)
    pos = m["pos"].clone()
    pos[:, ::3] = -1
    pos[1] = -7
    pad = pos < 0
    q, k = (torch.full(t.shape, 5.0, dtype=BF, device="cuda") for t in whole)
    attn.qk_norm_rope(m["q"], m["k"], cos, sin, positions=pos, q_out=q, k_out=k, **kw)
    dq, dk = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], positions=pos, dq=dq, dk=dk, **kw)
    for got, want in zip((q, k, dq, dk), whole + full[:2]):
        assert (got[pad] == 5.0).all() and torch.equal(got[~pad], want[~pad])
    # dw of the rows that are left, from the float64 form
    c, s = cos[pos.clamp(min=0).long()].double(), sin[pos.clamp(min=0).long()].double()
    for x, w, dz, dw in ((m["q"], m["wq"], m["dqo"], g[2]), (m["k"], m["wk"], m["dko"], g[3])):
        w64 = w.double().requires_grad_()
        z = kvref.norm_rope(x.double(), w64, c, s, True, 1e-6, False)
        ((z * dz.double())[~pad]).sum().backward()
        r = 1 / torch.sqrt(x.double().pow(2).mean(-1, keepdim=True) + 1e-6)
        total = (pair_length(dz.double(), 64, False) * (x.double() * r).abs())[~pad].sum((0, 1))
        close(dw, w64.grad, 2.0 ** -24 * (63 * x.shape[2] + 64) * total)


@pytest.mark.parametrize("heads,d", [((5, 2), 128), ((1, 1), 64), ((3, 1), 192)])
def test_gradient_without_eps(heads, d):
    """Lanes without a row add nothing to the weights' gradient, at eps = 0 either."""
    cos, sin = attn.rope_tables(5000, 64)
    check(make(2, 19, *heads, d, BF, seed=22, spread=False), cos, sin, False, eps=0.0)


def test_tables_without_positions():
    """max_pos = 0: every position is outside, and nothing is read."""
    m = make(1, 9, 4, 2, 128, BF, seed=23)
    cos, sin = (t[:0] for t in attn.rope_tables(8, 128))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, positions=m["pos"], status=status)
    except attn.AttnError:
        return  # (an empty tensor without an address is refused)
    assert torch.isnan(z[0]).all() and torch.isnan(z[1]).all()
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)


def special_rows(m, value, cos, sin, **kw):
    """`value` in one element of one query and one key row: outputs, gradients and
    their float64 forms (differentiated by autograd)."""
    at = {"q": (0, 3, 0, 7), "k": (1, 5, m["k"].shape[2] - 1, m["k"].shape[3] - 1)}
    for n, i in at.items():
        m[n][i] = value
    z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, positions=m["pos"], wq=m["wq"], wk=m["wk"], **kw)
    g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], positions=m["pos"], wq=m["wq"],
                              wk=m["wk"], **kw)
    c, s = cos[m["pos"].long()].double(), sin[m["pos"].long()].double()
    for n, got, w, dz, dx, dw in (("q", z[0], m["wq"], m["dqo"], g[0], g[2]), ("k", z[1], m["wk"], m["dko"], g[1], g[3])):
        x64, w64 = m[n].double().requires_grad_(), w.double().requires_grad_()
        want = kvref.norm_rope(x64, w64, c, s, True, kw.get("eps", 1e-6), False)
        (want * dz.double()).sum().backward()
        yield at[n], (got, want.detach()), (dx, x64.grad), (dw, w64.grad)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("heads,d", [((5, 2), 128), ((1, 1), 64), ((3, 1), 192), ((4, 4), 512)])
def test_nan_in_a_row(heads, d, dt):
    """A NaN makes its row NaN, forward and gradient, and all of dw; no other row
    changes."""
    cos, sin = attn.rope_tables(5000, 64)
    m = make(2, 11, *heads, d, dt, seed=24, spread=False)
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])
    clean = attn.qk_norm_rope(m["q"], m["k"], cos, sin, **kw)
    clean_g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)
    for i, (at, z, dx, dw) in enumerate(special_rows(m, float("nan"), cos, sin)):
        others = torch.ones(z[0].shape[:3], dtype=torch.bool)
        others[at[:3]] = False
        for (got, want), before in ((z, clean[i]), (dx, clean_g[i])):
            assert torch.isnan(want[~others]).all() and torch.isnan(got[~others]).all()
            assert torch.equal(got[others], before[others])
        assert torch.isnan(dw[1]).all() and torch.isnan(dw[0]).all()


@pytest.mark.parametrize("heads,d", [((5, 2), 128), ((1, 1), 64), ((3, 1), 192)])
def test_tiny_rows_without_eps(heads, d):
    """Rows of about 2^-64 at eps = 0, whose mean square 2^-128 is below FP32's
    normal range: a square or sum there is off by 2^-150 at most, 2^-22 of a mean
    square, so the bounds are twice those of ordinary rows.  Rows of zeros: zeros."""
    cos, sin = attn.rope_tables(5000, 64)
    m = make(2, 11, *heads, d, BF, seed=25, spread=False)
    for t in (m["q"], m["k"]):
        t.mul_(2.0 ** -64)
    m["q"][0, 0, 0] = 0.0
    zero = torch.zeros(2, 11, heads[0], dtype=torch.bool)
    zero[0, 0, 0] = True
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"], eps=0.0)
    z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, **kw)
    g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)
    assert (z[0][zero] == 0).all() and (g[0][zero] == 0).all()
    m["q"][0, 0, 0] = 1.0  # (for the float64 form)
    dz = m["dqo"].double()
    dz[0, 0, 0] = 0.0
    c, s = cos[m["pos"].long()].double(), sin[m["pos"].long()].double()
    u = UNIT[BF]
    for x, w, dz, got, dx, dw, skip in ((m["q"], m["wq"], dz, z[0], g[0], g[2], zero),
                                        (m["k"], m["wk"], m["dko"].double(), z[1], g[1], g[3], None)):
        live = slice(None) if skip is None else ~skip
        x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
        want = kvref.norm_rope(x64, w64, c, s, True, 0.0, False)
        length = pair_length(kvref.norm_rope(x64, w64, None, None, True, 0.0, False).detach(), 64, False)
        close(got[live], want.detach()[live], (u * want.detach().abs() + 2.0 ** -17 * length + 2.0 ** -25)[live])
        (want * dz).sum().backward()
        r = 1 / x.double().pow(2).mean(-1, keepdim=True).sqrt()
        gl = pair_length(dz, 64, False) * w.double().abs()
        size = r * (gl + x.double().abs() * r * r * (gl * x.double().abs()).mean(-1, keepdim=True))
        close(dx[live], x64.grad[live], (u * x64.grad.abs() + 2.0 ** -16 * size)[live])
        total = (gl / w.double().abs() * (x.double() * r).abs()).sum((0, 1, 2))
        close(dw, w64.grad, 2.0 ** -24 * (22 * x.shape[2] + 128) * total)


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("heads,d", [((5, 2), 128), ((1, 1), 64), ((3, 1), 192), ((4, 4), 512)])
def test_infinity_in_a_row(heads, d, dt, value):
    """With the norm an infinity becomes NaN, as what it is turned with does, and
    leaves zeros beside it; its row of dx is NaN, dw where the float64 form is."""
    cos, sin = attn.rope_tables(5000, 64)
    m = make(2, 11, *heads, d, dt, seed=24, spread=False)
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])
    clean = attn.qk_norm_rope(m["q"], m["k"], cos, sin, **kw)
    clean_g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)
    # |dy x r| of the untouched rows bounds what the sums of dw add up
    total = [(pair_length(dz.double(), 64, False) * x.double().abs()
              / x.double().pow(2).mean(-1, keepdim=True).sqrt()).sum((0, 1, 2))
             for x, dz in ((m["q"], m["dqo"]), (m["k"], m["dko"]))]
    for i, (at, z, dx, dw) in enumerate(special_rows(m, value, cos, sin)):
        row = at[:3]
        others = torch.ones(z[0].shape[:3], dtype=torch.bool)
        others[row] = False
        for (got, want), before in ((z, clean[i]), (dx, clean_g[i])):
            assert torch.equal(got[others], before[others])
            assert torch.equal(torch.isnan(got[row]), torch.isnan(want[row]))
            assert (got[row].nan_to_num() == 0).all()
        bad = torch.isnan(dw[1])
        assert torch.equal(torch.isnan(dw[0]), bad) and bad.any()
        close(dw[0][~bad], dw[1][~bad], 2.0 ** -24 * (22 * heads[i] + 64) * total[i][~bad])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 64), (192, 16), (64, 0), (256, 256)])
def test_elements_that_do_not_turn_do_not_meet(d, rot, inter):
    """Without the norm an infinity or a NaN reaches the element it is turned with
    and no other, forward and gradient."""
    cos, sin = attn.rope_tables(5000, rot) if rot else (None, None)
    m = make(1, 7, 3, 2, d, BF, seed=27, spread=False)
    kw = dict(positions=m["pos"], norm=False, interleaved=inter)
    c, s = (cos[m["pos"].long()].double(), sin[m["pos"].long()].double()) if rot else (None, None)
    for j in {0, 1, rot // 2, max(rot - 1, 0), min(rot, d - 1), d // 2, d - 9, d - 1}:
        for value in (float("inf"), float("nan")):
            x, dz = m["q"].clone(), m["dqo"].clone()
            x[0, 3, 1, j] = dz[0, 4, 2, j] = value
            z, _ = attn.qk_norm_rope(x, None, cos, sin, **kw)
            want = kvref.norm_rope(x.double(), None, c, s, False, 0.0, inter)
            dx, _, _, _ = attn.qk_norm_rope_bwd(m["q"], None, cos, sin, dz, None, **kw)
            grad = kvref.turn(dz.double(), c, s, inter, -1) if rot else dz.double()
            for got, ref in ((z, want), (dx, grad)):
                assert torch.equal(torch.isnan(got), torch.isnan(ref))
                assert torch.equal(torch.isinf(got), torch.isinf(ref))


@pytest.mark.parametrize("heads", [(5, 2), (1, 1)])
def test_gradient_without_norm_does_not_depend_on_x(heads):
    m = make(2, 11, *heads, 128, BF, seed=28, spread=False)
    cos, sin = attn.rope_tables(5000, 64)
    kw = dict(positions=m["pos"], norm=False)
    want = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)
    m["q"][0, 2, 0, 3], m["k"][1, 4, -1, 70], m["q"][1, 1] = float("inf"), float("nan"), 3e38
    got = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty_tables():
    """Tables of no rows: every position is outside, and nothing is read."""
    m = make(2, 9, 4, 2, 128, BF, seed=26)
    cos = sin = torch.empty(0, 64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m["pos"][0, 3] = -1
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])
    out = [torch.full(t.shape, 5.0, dtype=BF, device="cuda") for t in (m["q"], m["k"])]
    z = attn.qk_norm_rope(m["q"], m["k"], cos, sin, status=status, q_out=out[0], k_out=out[1], **kw)
    g = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)
    live = m["pos"] >= 0
    for t in (*z, g[0], g[1]):
        assert torch.isnan(t[live]).all()
    for t in z:
        assert (t[~live] == 5.0).all()
    assert torch.isnan(g[2]).all() and torch.isnan(g[3]).all()
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)


def test_tables_of_no_rows_are_not_read():
    """The C entry point with real addresses and max_pos = 0."""
    m = make(1, 9, 4, 2, 128, BF, seed=29)
    cos, sin = attn.rope_tables(16, 128)
    out = [torch.zeros_like(m[n], memory_format=torch.contiguous_format) for n in ("q", "k")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = attn.QkParams(0, 2, 1, 9, 4, 2, 128, 128, 0, 1, 0, 1e-6, m["q"].stride()[:3], m["k"].stride()[:3],
                      out[0].stride()[:3], out[1].stride()[:3])
    rc = attn.load().attn_qk_norm_rope(p, m["q"].data_ptr(), m["k"].data_ptr(), None, None, cos.data_ptr(),
                                       sin.data_ptr(), None, out[0].data_ptr(), out[1].data_ptr(),
                                       status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for t in out:
        assert torch.isnan(t).all()
    with pytest.raises(attn.AttnError, match="out of range"):
        attn.query_status(status)


@pytest.mark.parametrize("order", [(1, 0, 2), (0, 2, 1), (2, 0, 1)])
def test_in_place_in_other_layouts(order):
    """Views of one projection whose axes lie in another order, written in place."""
    m = make(3, 20, 4, 2, 64, BF, seed=30)
    cos, sin = attn.rope_tables(5000, 64)
    kw = dict(positions=m["pos"], wq=m["wq"], wk=m["wk"])
    want = attn.qk_norm_rope(m["q"], m["k"], cos, sin, **kw)
    grad = attn.qk_norm_rope_bwd(m["q"], m["k"], cos, sin, m["dqo"], m["dko"], **kw)

    def merged(a, b):  # both as views of one buffer [.. in that order .., d]
        x = torch.cat((a, b, b), 2).permute(*order, 3).contiguous().permute(*(order.index(i) for i in range(3)), 3)
        return x, x[:, :, :4], x[:, :, 4:6]

    x, q, k = merged(m["q"], m["k"])
    rest = x[:, :, 6:].clone()
    g, dq, dk = merged(m["dqo"], m["dko"])
    got = attn.qk_norm_rope_bwd(q, k, cos, sin, dq, dk, dq=dq, dk=dk, **kw)
    for a, b in zip(got, grad):
        assert torch.equal(a, b)
    attn.qk_norm_rope(q, k, cos, sin, q_out=q, k_out=k, **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, :, 6:], rest)
