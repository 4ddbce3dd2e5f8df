"""Arguments that the operators around the attention kernels refuse (no GPU:
every call here is refused before anything is launched), their workspace sizes,
and pins of the float64 forms in kvref.py."""
import ctypes

import pytest
import torch

import kvref
from bwd_tcgen05_tmem_gb300 import attn, build

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load()


def at(mb, off=0):
    return ctypes.c_void_p(mb * MB + off)


# ------------------------------------------------------------------ norm and rotation

def qk_params(**kw):
    b, s, hq, hk, d = 2, 100, 4, 2, 128
    st_q, st_k = (s * hq * d, hq * d, d), (s * hk * d, hk * d, d)
    p = attn.QkParams(0, 2, b, s, hq, hk, d, 128, 0, 1, 4096, 1e-6, st_q, st_k, st_q, st_k, st_q, st_k)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(p, k)[:] = v
        else:
            setattr(p, k, v)
    return p


def qk_call(lib, p, bwd=False, **ptrs):
    a = dict(q=at(64), k=at(128), wq=at(1), wk=at(2), cos=at(10), sin=at(20), pos=at(3),
             dqo=at(192), dko=at(256), qo=at(320), ko=at(384), dwq=at(4), dwk=at(5), ws=at(512),
             status=at(6), nbytes=64 * MB)
    a.update(ptrs)
    if bwd:
        return lib.attn_qk_norm_rope_bwd(p, a["q"], a["k"], a["wq"], a["wk"], a["cos"], a["sin"],
                                         a["pos"], a["dqo"], a["dko"], a["qo"], a["ko"], a["dwq"],
                                         a["dwk"], a["ws"], a["nbytes"], a["status"], None)
    return lib.attn_qk_norm_rope(p, a["q"], a["k"], a["wq"], a["wk"], a["cos"], a["sin"], a["pos"],
                                 a["qo"], a["ko"], a["status"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("change,ptrs,code", [
    (dict(dtype=2), {}, UNSUPPORTED), (dict(w_dtype=1), {}, UNSUPPORTED),
    (dict(head_dim=96), {}, UNSUPPORTED), (dict(rotary_dim=24), {}, UNSUPPORTED),
    (dict(rotary_dim=144), {}, UNSUPPORTED), (dict(batch=-1), {}, INVALID),
    (dict(heads_q=0), {}, INVALID), (dict(heads_k=-1), {}, INVALID),
    (dict(eps=float("nan")), {}, INVALID), (dict(eps=-1.0), {}, INVALID),
    (dict(max_pos=-1), {}, INVALID), (dict(norm=0), {}, INVALID),
    (dict(batch=1 << 20, seqlen=1 << 20), {}, UNSUPPORTED),
    (dict(stride_q=(51200, 516, 128)), {}, ALIGN), (dict(stride_q=(-8, 512, 128)), {}, INVALID),
    (dict(stride_qo=(51200, 512, 64)), {}, INVALID),  # heads of the output share memory
    (dict(stride_qo=(0, 512, 128)), {}, INVALID),     # so do its sequences
    ({}, dict(q=None), INVALID), ({}, dict(q=at(64, 8)), ALIGN), ({}, dict(qo=at(320, 2)), ALIGN),
    ({}, dict(cos=None), INVALID), ({}, dict(sin=at(20, 4)), ALIGN), ({}, dict(wq=at(1, 4)), ALIGN),
    ({}, dict(pos=at(3, 2)), ALIGN), ({}, dict(status=at(6, 1)), ALIGN),
    ({}, dict(qo=at(128)), INVALID),          # over k
    ({}, dict(qo=at(64, 1024)), INVALID),     # over q, shifted
    ({}, dict(qo=at(384)), INVALID),          # over the output of k
    ({}, dict(ko=at(10)), INVALID),           # over the cosines
    ({}, dict(ko=at(3)), INVALID),            # over the positions
])
def test_qk_refusals(lib, bwd, change, ptrs, code):
    assert qk_call(lib, qk_params(**change), bwd, **ptrs) == code
    assert lib.attn_last_error()


@pytest.mark.parametrize("change,ptrs,code", [
    ({}, dict(ws=None), WORKSPACE), ({}, dict(ws=at(512, 64)), ALIGN), ({}, dict(nbytes=16), WORKSPACE),
    ({}, dict(wq=None), INVALID),             # a gradient of absent weights
    ({}, dict(qo=at(64)), INVALID),           # dq over q
    ({}, dict(dwq=at(512)), INVALID),         # dw inside the workspace
    ({}, dict(dwk=at(4)), INVALID),           # dw_q over dw_k
    ({}, dict(dqo=None), INVALID), ({}, dict(dwq=at(4, 2)), ALIGN),
])
def test_qk_backward_refusals(lib, change, ptrs, code):
    assert qk_call(lib, qk_params(**change), True, **ptrs) == code


def test_qk_slices_of_one_buffer_do_not_overlap(lib):
    """q and k as slices of one projection, written in place: the rows interleave
    and share no element; one element more and they do.  (A refused argument
    behind the overlap checks shows that they passed.)"""
    d, h = 128, 8
    st = (100 * h * d, h * d, d)
    p = qk_params(stride_q=st, stride_k=st, stride_qo=st, stride_ko=st)
    k = at(64, 4 * d * 2)  # heads 4, 5 of 8
    table = at(64, 6 * d * 2)  # the cosines lie in the buffer's heads 6, 7: refused last
    assert qk_call(lib, p, q=at(64), k=k, qo=at(64), ko=k, cos=table) == INVALID
    assert b"tables" in lib.attn_last_error()
    k = at(64, 4 * d * 2 - 16)
    assert qk_call(lib, p, q=at(64), k=k, qo=at(64), ko=k, cos=table) == INVALID
    assert b"tables" not in lib.attn_last_error()


def test_qk_nothing_to_do(lib):
    assert qk_call(lib, qk_params(seqlen=0)) == OK
    assert lib.attn_last_launch_count() == 0


def test_qk_workspace_is_a_partial_sum_for_each_block(lib):
    p = qk_params(seqlen=1, batch=1)
    # one token: a block for each side at least, 128 floats each, in 256-byte steps
    assert lib.attn_qk_norm_rope_bwd_workspace_size(p) == 2 * 128 * 4
    assert lib.attn_qk_norm_rope_bwd_workspace_size(qk_params(head_dim=96)) == 256


# ------------------------------------------------------------------ page plan

def plan_call(lib, change=(), **ptrs):
    p = attn.KvPlanParams(4, 8, 64, 100, 50, 30, 8)
    for k, v in dict(change).items():
        setattr(p, k, v)
    a = dict(ctx=at(1), fresh=at(2), table=at(3), free=at(4), head=at(5), cu=at(6), seq=at(7), pos=at(8),
             slots=at(9), head_out=at(10), status=at(11))
    a.update(ptrs)
    return lib.attn_kv_plan(p, *a.values(), None)


@pytest.mark.parametrize("change,ptrs,code", [
    (dict(batch=-1), {}, INVALID), (dict(batch=8193), {}, UNSUPPORTED), (dict(page_size=48), {}, UNSUPPORTED),
    (dict(page_size=8), {}, UNSUPPORTED), (dict(page_size=512), {}, UNSUPPORTED),
    (dict(page_size=0), {}, UNSUPPORTED), (dict(rows=-1), {}, INVALID), (dict(n_free=-1), {}, INVALID),
    (dict(cols=1 << 25), {}, UNSUPPORTED), (dict(num_pages=1 << 26), {}, UNSUPPORTED),
    (dict(table_stride=7), {}, INVALID),
    ({}, dict(ctx=None), INVALID), ({}, dict(table=None), INVALID), ({}, dict(head=None), INVALID),
    ({}, dict(head_out=None), INVALID), ({}, dict(cu=None), INVALID), ({}, dict(slots=None), INVALID),
    ({}, dict(pos=at(8, 1)), ALIGN), ({}, dict(status=at(11, 2)), ALIGN),
    ({}, dict(seq=at(1)), INVALID), ({}, dict(head_out=at(5)), INVALID), ({}, dict(slots=at(8)), INVALID),
    ({}, dict(cu=at(3, 4)), INVALID),
])
def test_plan_refusals(lib, change, ptrs, code):
    assert plan_call(lib, change.items(), **ptrs) == code


# ------------------------------------------------------------------ the cache

def cache_desc(**kw):
    c = attn.Kv4CacheDesc(100 * MB, 200 * MB, 300 * MB, 400 * MB, 50, 64, 2, 128, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("name", ["attn_kv_write", "attn_kv_read"])
@pytest.mark.parametrize("change,args,code", [
    (dict(d_qk=96), {}, UNSUPPORTED), (dict(d_qk=512, d_v=512), {}, UNSUPPORTED),
    (dict(d_v=64), {}, UNSUPPORTED), (dict(page_size=24), {}, UNSUPPORTED), (dict(heads_kv=0), {}, INVALID),
    (dict(num_pages=1 << 25), {}, UNSUPPORTED), (dict(num_pages=-1), {}, INVALID),
    (dict(k_codes=None), {}, INVALID), (dict(v_scales=400 * MB + 2), {}, ALIGN),
    ({}, dict(dtype=2), UNSUPPORTED), ({}, dict(tokens=-1), INVALID), ({}, dict(k=None), INVALID),
    ({}, dict(v=at(12, 4)), ALIGN), ({}, dict(sk=(260, 128)), ALIGN), ({}, dict(sk=(-256, 128)), INVALID),
    ({}, dict(sk=None), INVALID), ({}, dict(slots=None), INVALID), ({}, dict(slots=at(2, 1)), ALIGN),
    ({}, dict(k=at(100)), INVALID), ({}, dict(v=at(399, 1 << 19), sv=(1 << 15, 128)), INVALID),
    (dict(heads_kv=65536), dict(tokens=1 << 20), UNSUPPORTED),
])
def test_cache_rows_refusals(lib, name, change, args, code):
    a = dict(dtype=0, tokens=40, k=at(10), sk=(256, 128), v=at(12), sv=(256, 128), slots=at(2), status=at(3))
    a.update(args)
    pair = ctypes.c_int64 * 2
    st = [pair(*a[x]) if a[x] else None for x in ("sk", "sv")]
    rc = getattr(lib, name)(cache_desc(**change), a["dtype"], a["tokens"], a["k"], st[0], a["v"], st[1],
                            a["slots"], a["status"], None)
    assert rc == code


def test_cache_read_outputs_must_not_share_memory(lib):
    pair = ctypes.c_int64 * 2
    wide, none = pair(256, 128), pair(0, 128)
    assert lib.attn_kv_read(cache_desc(), 0, 40, at(10), none, at(12), wide, at(2), None, None) == INVALID
    assert lib.attn_kv_read(cache_desc(), 0, 40, at(10), wide, at(10, 256), wide, at(2), None, None) == INVALID
    assert lib.attn_kv_write(cache_desc(v_codes=100 * MB), 0, 40, at(10), wide, at(12), wide, at(2), None,
                              None) == INVALID


def decode_params(**kw):
    st = (4 * 128, 4 * 128, 128)
    p = attn.Kv4DecodeParams(0, 0, 3, 1, 4, st, st, 16, 16, -1, 0, 0.1)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(p, k)[:] = v
        else:
            setattr(p, k, v)
    return p


@pytest.mark.parametrize("change,cache,ptrs,code", [
    (dict(dtype=2), {}, {}, UNSUPPORTED), (dict(o_dtype=1), {}, {}, UNSUPPORTED),
    (dict(batch=-1), {}, {}, INVALID), (dict(seqlen_q=257), {}, {}, UNSUPPORTED),
    (dict(seqlen_q=-1), {}, {}, INVALID), (dict(heads_q=3), {}, {}, INVALID),
    (dict(heads_q=0), {}, {}, INVALID), (dict(heads_q=2 * 129), {}, {}, UNSUPPORTED),
    (dict(cols=1 << 25), {}, {}, UNSUPPORTED), (dict(table_stride=-1), {}, {}, INVALID),
    (dict(window_left=-2), {}, {}, INVALID), (dict(sinks=-1), {}, {}, INVALID),
    (dict(softmax_scale=0.0), {}, {}, INVALID), (dict(softmax_scale=float("inf")), {}, {}, INVALID),
    (dict(stride_q=(512, 512, 4)), {}, {}, ALIGN), (dict(stride_o=(512, 512, 64)), {}, {}, INVALID),
    ({}, dict(d_qk=512, d_v=512), {}, UNSUPPORTED), ({}, dict(page_size=8), {}, UNSUPPORTED),
    ({}, dict(k_scales=None), {}, INVALID),
    ({}, {}, dict(q=None), INVALID), ({}, {}, dict(q=at(10, 2)), ALIGN), ({}, {}, dict(lse=None), INVALID),
    ({}, {}, dict(lens=None), INVALID), ({}, {}, dict(table=None), INVALID), ({}, {}, dict(ws=None), WORKSPACE),
    ({}, {}, dict(nbytes=256), WORKSPACE), ({}, {}, dict(ws=at(500, 16)), ALIGN),
    ({}, {}, dict(o=at(10)), INVALID), ({}, {}, dict(o=at(500)), INVALID), ({}, {}, dict(lse=at(3)), INVALID),
    ({}, {}, dict(ws=at(100)), INVALID),
])
def test_decode_refusals(lib, change, cache, ptrs, code):
    a = dict(q=at(10), table=at(2), lens=at(3), o=at(12), lse=at(14), ws=at(500), nbytes=64 * MB, status=at(4))
    a.update(ptrs)
    assert lib.attn_kv_decode(decode_params(**change), cache_desc(**cache), *a.values(), None) == code


def test_decode_nothing_to_do(lib):
    ws = dict(q=None, table=None, lens=None, o=None, lse=None, ws=at(500), nbytes=64 * MB, status=None)
    assert lib.attn_kv_decode(decode_params(batch=0), cache_desc(), *ws.values(), None) == OK
    assert lib.attn_kv_decode(decode_params(seqlen_q=0), cache_desc(), *ws.values(), None) == OK


def test_decode_workspace_does_not_grow_with_the_context(lib):
    """Two partial results a run, whatever the lengths: only a few bytes an item
    grow with the batch."""
    size = lambda **kw: lib.attn_kv_decode_workspace_size(decode_params(**kw), cache_desc())  # noqa: E731
    long, longer = size(batch=64, cols=1 << 10), size(batch=64, cols=1 << 14)
    assert long == longer
    assert 0 < size(batch=128, cols=1 << 10) - long <= 64 * 2 * 8
    assert size(dtype=2) == 256


def test_python_refusals():
    q = torch.empty(2, 5, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attn.qk_norm_rope(q, q, None, None)


# ------------------------------------------------------------------ the float64 forms

def test_reference_codes_are_a_permutation_of_the_nibbles():
    g = torch.Generator().manual_seed(1)
    for d in (64, 128, 192, 256):
        for is_k in (True, False):
            c = torch.randint(0, 16, (3, d), generator=g)
            assert torch.equal(kvref.unpack(kvref.pack(c, is_k), is_k), c)


def test_reference_layout_by_hand():
    """G = 4: K word c * 4 + g, V half-word r * 4 + g; lowest nibble first."""
    one = torch.zeros(128, dtype=torch.int64)
    one[32 * 2 + 8 * 3 + 5] = 9      # K: word 3 * 4 + 2 = 14, nibble 5: byte 58, high half
    b = kvref.pack(one, True)
    assert b[58] == 9 << 4 and int(b.sum()) == 9 << 4
    one = torch.zeros(128, dtype=torch.int64)
    one[32 * 1 + 4 * 6 + 2] = 5      # V: half-word 6 * 4 + 1 = 25, nibble 2: byte 51, low half
    b = kvref.pack(one, False)
    assert b[51] == 5 and int(b.sum()) == 5


def test_reference_rotation_gradient_is_its_transpose():
    g = torch.Generator().manual_seed(2)
    ang = torch.randn(7, 8, generator=g, dtype=torch.float64)
    for inter in (False, True):
        y = torch.randn(7, 3, 32, generator=g, dtype=torch.float64, requires_grad=True)
        z = torch.randn(7, 3, 32, generator=g, dtype=torch.float64)
        (kvref.turn(y, ang.cos(), ang.sin(), inter) * z).sum().backward()
        assert torch.allclose(y.grad, kvref.turn(z, ang.cos(), ang.sin(), inter, -1), atol=1e-13)


def test_reference_norm_rope_by_hand():
    x = torch.zeros(1, 1, 64, dtype=torch.float64)
    x[..., 0], x[..., 1], x[..., 32] = 3.0, 4.0, 12.0
    r = (169.0 / 64 + 0.0) ** -0.5
    cos, sin = torch.zeros(1, 32, dtype=torch.float64), torch.ones(1, 32, dtype=torch.float64)
    z = kvref.norm_rope(x, None, cos, sin, True, 0.0, False)  # a quarter turn of (0, 32), (1, 33)
    assert torch.allclose(z[0, 0, [0, 32, 33]], torch.tensor([-12.0, 3.0, 4.0], dtype=torch.float64) * r)
    z = kvref.norm_rope(x, None, cos, sin, True, 0.0, True)   # of (0, 1)
    assert torch.allclose(z[0, 0, [0, 1]], torch.tensor([-4.0, 3.0], dtype=torch.float64) * r)


def test_reference_norm_rope_gradient_against_differences():
    """autograd of the float64 form, which the GPU gradients are held to, equals
    central differences (and so does the formula that the kernel evaluates)."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    ang = r(5, 8)
    for inter in (False, True):
        x, w = r(5, 2, 64).requires_grad_(), r(64).requires_grad_()
        f = lambda x, w: kvref.norm_rope(x, w, ang.cos(), ang.sin(), True, 1e-3, inter)  # noqa: E731
        assert torch.autograd.gradcheck(f, (x, w), eps=1e-6, atol=1e-7)
        dz = r(5, 2, 64)
        dx, dw = torch.autograd.grad((f(x, w) * dz).sum(), (x, w))
        n = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + 1e-3)
        dy = kvref.turn(dz, ang.cos(), ang.sin(), inter, -1)
        e = dy * w
        assert torch.allclose(dw, (dy * x * n).sum((0, 1)), atol=1e-12)
        assert torch.allclose(dx, n * (e - x * n * n * (e * x).mean(-1, keepdim=True)), atol=1e-12)


def test_packed_parameters_are_the_structs():
    """The bytes that the bindings pass are those of the ctypes mirrors."""
    import random
    r = random.Random(1)
    for pack, struct, floats in ((attn._QK_PACK, attn.QkParams, (11,)), (attn._PLAN_PACK, attn.KvPlanParams, ()),
                                 (attn._DECODE_PACK, attn.Kv4DecodeParams, (15,))):
        flat = [n for _, t in struct._fields_ for n in range(getattr(t, "_length_", 1))]
        vals = [0.5 if i in floats else r.randrange(1, 1 << 20) for i in range(len(flat))]
        it = iter(vals)
        args = [tuple(next(it) for _ in range(t._length_)) if hasattr(t, "_length_") else next(it)
                for _, t in struct._fields_]
        got, want = struct.from_buffer_copy(pack(*vals)), struct(*args)
        for name, t in struct._fields_:
            a, b = getattr(got, name), getattr(want, name)
            assert list(a) == list(b) if hasattr(t, "_length_") else a == b, name
        assert len(pack(*vals)) == ctypes.sizeof(struct)


@pytest.mark.parametrize("call", ["plan", "write", "read", "decode", "qk", "qk_bwd"])
def test_python_refuses_status_words_and_workspaces_of_other_shapes(call):
    """The kernels write four bytes at the status' address and whole bytes from the
    workspace's on (looked at first, so no GPU is needed)."""
    from bwd_tcgen05_tmem_gb300 import kv
    ints, x = torch.zeros(4, dtype=torch.int32), torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    f = dict(plan=lambda **kw: kv.plan(ints, ints, ints.view(4, 1), page_size=16, num_pages=1, rows=1, **kw),
             write=lambda **kw: kv.kv4_write(None, x[0], x[0], ints, **kw),
             read=lambda **kw: kv.kv4_read(None, ints, k=x[0], v=x[0], **kw),
             decode=lambda **kw: kv.kv4_decode(x, None, ints, ints, **kw),
             qk=lambda **kw: attn.qk_norm_rope(x, x, None, None, **kw),
             qk_bwd=lambda **kw: attn.qk_norm_rope_bwd(x, x, None, None, x, x, **kw))[call]
    for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="status"):
            f(status=bad)
    if call in ("decode", "qk_bwd"):
        with pytest.raises(ValueError, match="workspace"):
            f(workspace=torch.zeros(1 << 16, dtype=torch.uint8)[::2])


def qk_overlap(lib, q, qs, q_out, os, shape, k=None, ks=None, k_out=None, kos=None, hk=0):
    """What refuses a call whose outputs lie where its tables do, which is looked at
    last: the tables, if everything else is apart (so nothing is ever launched)."""
    b, s, hq, d = shape
    st = lambda x: x or (0, 0, 0)  # noqa: E731
    p = attn.QkParams(0, 2, b, s, hq, hk, d, d, 0, 1, 4096, 1e-6, st(qs), st(ks), st(os), st(kos))
    rc = qk_call(lib, p, q=q, k=k, wq=None, wk=None, pos=None, qo=q_out, ko=k_out, cos=q_out, status=None)
    assert rc == INVALID
    return b"tables" not in lib.attn_last_error()


@pytest.mark.parametrize("layout", ["bshd", "sbhd", "bhsd", "hbsd", "shbd", "hsbd"])
def test_qk_slices_of_one_buffer_in_any_layout(lib, layout):
    """Slices along one axis of a buffer are apart, in whatever order its axes lie;
    in place they are the same; one vector of 8 elements further they overlap."""
    size = dict(b=3, s=50, h=8)
    stride, at_end = {}, 64
    for a in reversed(layout[:3]):
        stride[a], at_end = at_end, at_end * size[a]
    st = tuple(stride[a] for a in "bsh")
    base = 64 * MB
    ptr = lambda el: ctypes.c_void_p(base + 2 * el)  # noqa: E731
    # q heads 0 .. 3, k heads 4, 5, each in place
    k = ptr(4 * stride["h"])
    assert not qk_overlap(lib, ptr(0), st, ptr(0), st, (3, 50, 4, 64), k, st, k, st, 2)
    k = ptr(4 * stride["h"] - 8)
    assert qk_overlap(lib, ptr(0), st, ptr(0), st, (3, 50, 4, 64), k, st, k, st, 2)
    # half of the tokens into the others, one sequence into the next
    assert not qk_overlap(lib, ptr(0), st, ptr(25 * stride["s"]), st, (3, 25, 8, 64))
    assert qk_overlap(lib, ptr(0), st, ptr(24 * stride["s"]), st, (3, 25, 8, 64))
    assert not qk_overlap(lib, ptr(0), st, ptr(stride["b"]), st, (1, 50, 8, 64))
    # (sequences 2 and 3 of 3: the last one is behind the buffer, or the next token's or
    # head's first one, which the output holds)
    assert qk_overlap(lib, ptr(2 * stride["b"]), st, ptr(0), st, (2, 50, 8, 64)) == (layout[0] != "b")


def test_qk_overlaps_are_never_missed(lib):
    """Against the set of vectors of 8 elements that the tensors hold."""
    import random
    r = random.Random(7)
    apart = 0
    for _ in range(1500):
        shape = tuple(r.randint(1, 4) for _ in range(3))

        def tensor(output):
            order, st, inner = r.sample(range(3), 3), [0] * 3, 8
            for a in order:
                st[a] = inner * 8 * r.choice((1, 1, 1, 2, 3))
                inner = st[a] // 8 * shape[a]
                if not output and r.random() < 0.15:
                    st[a] = 0
            base = r.randrange(0, 2000) * 8
            held = {(base + i * st[0] + j * st[1] + h * st[2]) // 8 + e for i in range(shape[0])
                    for j in range(shape[1]) for h in range(shape[2]) for e in range(8)}
            return tuple(st), base, held

        (qs, qb, held), (os, ob, out) = tensor(False), tensor(True)
        if qb == ob and qs == os:
            continue
        got = qk_overlap(lib, ctypes.c_void_p(64 * MB + 2 * qb), qs, ctypes.c_void_p(64 * MB + 2 * ob), os, (*shape, 64))
        assert got or not held & out
        apart += not got
    assert apart > 300
