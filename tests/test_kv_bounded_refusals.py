"""Arguments that the operators on a shared and bounded cache refuse (no GPU: every call
here is refused before anything is launched), their workspace sizes, and pins of the
float64 forms in boundedref.py."""
import ctypes
import math
import random

import pytest
import torch

import boundedref
import kvref
from bwd_tcgen05_tmem_gb300 import attn, build, kv
from test_kv_refusals import ALIGN, INVALID, MB, OK, UNSUPPORTED, WORKSPACE, at, cache_desc, decode_params


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load()


def fill(p, kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(p, k)[:] = v
        else:
            setattr(p, k, v)
    return p


# ------------------------------------------------------------------ shared prefixes

def shared_call(lib, change=(), cache=(), groups=2, **ptrs):
    a = dict(starts=at(5), shared=at(6), q=at(10), table=at(2), lens=at(3), o=at(12), lse=at(14), ws=at(500),
             nbytes=256 * MB, status=at(4))
    a.update(ptrs)
    return lib.attn_kv_decode_shared(decode_params(**dict(change)), cache_desc(**dict(cache)), groups, *a.values(), None)


@pytest.mark.parametrize("change,cache,ptrs,code", [
    (dict(dtype=2), {}, {}, UNSUPPORTED), (dict(o_dtype=1), {}, {}, UNSUPPORTED), (dict(batch=-1), {}, {}, INVALID),
    (dict(seqlen_q=257), {}, {}, UNSUPPORTED), (dict(heads_q=3), {}, {}, INVALID),
    (dict(window_left=100), {}, {}, UNSUPPORTED), (dict(window_left=0), {}, {}, UNSUPPORTED),
    (dict(softmax_scale=-1.0), {}, {}, INVALID), (dict(stride_q=(512, 512, 4)), {}, {}, ALIGN),
    (dict(stride_o=(512, 512, 64)), {}, {}, INVALID), ({}, dict(d_qk=512, d_v=512), {}, UNSUPPORTED),
    ({}, dict(v_scales=None), {}, INVALID), ({}, {}, dict(groups=-1), INVALID), ({}, {}, dict(groups=4), INVALID),
    ({}, {}, dict(starts=None), INVALID), ({}, {}, dict(shared=None), INVALID), ({}, {}, dict(starts=at(5, 2)), ALIGN),
    ({}, {}, dict(q=None), INVALID), ({}, {}, dict(lse=None), INVALID), ({}, {}, dict(table=None), INVALID),
    ({}, {}, dict(ws=None), WORKSPACE), ({}, {}, dict(nbytes=MB), WORKSPACE), ({}, {}, dict(ws=at(500, 16)), ALIGN),
    ({}, {}, dict(o=at(10)), INVALID), ({}, {}, dict(o=at(510)), INVALID), ({}, {}, dict(lse=at(5)), INVALID),
    ({}, {}, dict(lse=at(6)), INVALID), ({}, {}, dict(ws=at(100)), INVALID), ({}, {}, dict(status=at(4, 2)), ALIGN),
])
def test_shared_refusals(lib, change, cache, ptrs, code):
    assert shared_call(lib, change, cache, **ptrs) == code
    assert lib.attn_last_error()


def test_shared_too_many_tiles(lib):
    """Tiles of query rows times tiles of keys are counted in 32 bits."""
    size, c = lib.attn_kv_decode_shared_workspace_size, cache_desc(num_pages=2 ** 20)
    few = dict(batch=4096, cols=2 ** 18, table_stride=2 ** 18)
    assert size(decode_params(**few), c, 2) > MB
    assert size(decode_params(**few, seqlen_q=256), c, 2) == 256  # (what a refused call is told)
    assert shared_call(lib, dict(few, seqlen_q=256), dict(num_pages=2 ** 20)) == UNSUPPORTED
    assert "too many tiles" in str(lib.attn_last_error())


def test_shared_nothing_to_do(lib):
    none = dict(starts=None, shared=None, q=None, table=None, lens=None, o=None, lse=None, status=None)
    assert shared_call(lib, dict(batch=0), groups=0, **none) == OK
    assert shared_call(lib, dict(seqlen_q=0), **none) == OK


def test_shared_workspace(lib):
    """A part for each query row, whatever the lengths; 256 bytes for what is refused."""
    size = lambda groups=1, **kw: lib.attn_kv_decode_shared_workspace_size(decode_params(**kw), cache_desc(), groups)  # noqa: E731
    small, large = size(batch=64, cols=1 << 10), size(batch=64, cols=1 << 14)
    assert small == large
    row = 3 * 128 * 4 + 2 * 8 + 4
    more = size(batch=128, cols=1 << 10) - small
    assert 64 * 4 * row <= more <= 64 * (4 * row + 64) + 4096
    assert size(dtype=2) == 256 and size(groups=-1) == 256


# ------------------------------------------------------------------ weights

def weights_params(**kw):
    st = (4 * 128, 4 * 128, 128)
    return fill(attn.Kv4WeightsParams(0, 3, 1, 4, st, 16, 16, -1, 0, 0.1, 1, 1000, (2000, 1000)), kw)


@pytest.mark.parametrize("change,cache,ptrs,code", [
    (dict(dtype=2), {}, {}, UNSUPPORTED), (dict(batch=-1), {}, {}, INVALID), (dict(seqlen_q=257), {}, {}, UNSUPPORTED),
    (dict(heads_q=3), {}, {}, INVALID), (dict(heads_q=2 * 129), {}, {}, UNSUPPORTED),
    (dict(cols=1 << 25), {}, {}, UNSUPPORTED), (dict(table_stride=-1), {}, {}, INVALID),
    (dict(window_left=-2), {}, {}, INVALID), (dict(sinks=-1), {}, {}, INVALID), (dict(softmax_scale=0.0), {}, {}, INVALID),
    (dict(capacity=-1), {}, {}, INVALID), (dict(stride_w=(2000, -1)), {}, {}, INVALID),
    (dict(stride_w=(2000, 999)), {}, {}, INVALID), (dict(stride_w=(1999, 1000)), {}, {}, INVALID),
    (dict(stride_w=(0, 1000)), {}, {}, INVALID), (dict(stride_w=(1000, 2999)), {}, {}, INVALID),
    (dict(stride_q=(512, 512, 4)), {}, {}, ALIGN), ({}, dict(page_size=8), {}, UNSUPPORTED),
    ({}, {}, dict(q=None), INVALID), ({}, {}, dict(lse=None), INVALID), ({}, {}, dict(w=None), INVALID),
    ({}, {}, dict(w=at(14, 2)), ALIGN), ({}, {}, dict(lens=None), INVALID), ({}, {}, dict(table=None), INVALID),
    ({}, {}, dict(w=at(10)), INVALID), ({}, {}, dict(w=at(12)), INVALID), ({}, {}, dict(w=at(100)), INVALID),
    ({}, {}, dict(w=at(3)), INVALID), ({}, {}, dict(status=at(14)), INVALID),
])
def test_weights_refusals(lib, change, cache, ptrs, code):
    a = dict(q=at(10), table=at(2), lens=at(3), lse=at(12), w=at(14), status=at(4))
    a.update(ptrs)
    assert lib.attn_kv_weights(weights_params(**change), cache_desc(**cache), *a.values(), None) == code
    assert lib.attn_last_error()


def test_weights_nothing_to_do(lib):
    none = [None] * 7
    assert lib.attn_kv_weights(weights_params(batch=0), cache_desc(), *none) == OK
    assert lib.attn_kv_weights(weights_params(seqlen_q=0), cache_desc(), *none) == OK


def test_weights_of_no_queries_are_set_to_something(lib):
    """Without queries, accumulate = 0 still writes: what it writes to is checked, q and lse are not needed."""
    a = dict(q=None, table=at(2), lens=at(3), lse=None, w=at(14), status=at(4))
    for change in (dict(w=None), dict(lens=None), dict(table=None), dict(w=at(2)), dict(w=at(100)), dict(status=at(14))):
        args = {**a, **change}.values()
        assert lib.attn_kv_weights(weights_params(seqlen_q=0, accumulate=0), cache_desc(), *args, None) == INVALID


# ------------------------------------------------------------------ eviction

def evict_params(**kw):
    return fill(attn.Kv4EvictParams(3, 16, 16, 100, 10, 1000, (2000, 1000), (2000, 1000), 50), kw)


@pytest.mark.parametrize("change,cache,ptrs,code", [
    (dict(batch=-1), {}, {}, INVALID), (dict(keep=0), {}, {}, INVALID), (dict(recent=-1), {}, {}, INVALID),
    (dict(capacity=-1), {}, {}, INVALID), (dict(n_free=-1), {}, {}, INVALID), (dict(cols=1 << 25), {}, {}, UNSUPPORTED),
    (dict(keep=(1 << 30) + 1), {}, {}, UNSUPPORTED), (dict(batch=1 << 24), {}, {}, UNSUPPORTED),
    (dict(table_stride=-1), {}, {}, INVALID), (dict(stride_wo=(2000, 999)), {}, {}, INVALID),
    ({}, dict(page_size=24), {}, UNSUPPORTED), ({}, dict(k_codes=None), {}, INVALID),
    ({}, {}, dict(w=None), INVALID), ({}, {}, dict(w_out=None), INVALID), ({}, {}, dict(kept=None), INVALID),
    ({}, {}, dict(lens=None), INVALID), ({}, {}, dict(lens_out=None), INVALID), ({}, {}, dict(table=None), INVALID),
    ({}, {}, dict(first=at(7, 2)), ALIGN), ({}, {}, dict(w_out=at(14, 4)), INVALID),   # over the weights, shifted
    (dict(stride_wo=(1000, 3000)), {}, {}, INVALID),                                   # over them in another order
    ({}, {}, dict(lens_out=at(3)), INVALID), ({}, {}, dict(kept=at(14)), INVALID), ({}, {}, dict(kept=at(2)), INVALID),
    ({}, {}, dict(head_out=at(9)), INVALID), ({}, {}, dict(head_out=None), INVALID), ({}, {}, dict(free=None), INVALID),
    ({}, {}, dict(free=at(9)), INVALID), ({}, {}, dict(kept=at(100)), INVALID), ({}, {}, dict(first=at(16)), INVALID),
    ({}, dict(v_codes=100 * MB), {}, INVALID),  # the cache's arrays overlap
    ({}, {}, dict(status=at(4, 1)), ALIGN),
])
def test_evict_refusals(lib, change, cache, ptrs, code):
    a = dict(table=at(2), lens=at(3), first=at(7), w=at(14), w_out=at(14), kept=at(16), lens_out=at(5), free=at(8),
             head=at(9), head_out=at(11), status=at(4))
    a.update(ptrs)
    assert lib.attn_kv_evict(evict_params(**change), cache_desc(**cache), *a.values(), None) == code
    assert lib.attn_last_error()


def test_evict_refuses_more_sequences_than_a_free_list_takes(lib):
    """Each sequence adds up the pages of all: the time grows with the batch's square."""
    many = evict_params(batch=2 ** 16 + 1, cols=1, table_stride=1)
    a = dict(table=at(2), lens=at(3), first=at(7), w=at(14), w_out=at(14), kept=at(16), lens_out=at(5), free=at(8),
             head=at(9), head_out=at(11), status=at(4))
    assert lib.attn_kv_evict(many, cache_desc(), *a.values(), None) == UNSUPPORTED
    assert "2^16 sequences" in str(lib.attn_last_error())


def test_evict_nothing_to_do(lib):
    assert lib.attn_kv_evict(evict_params(batch=0), cache_desc(), *[None] * 12) == OK


# ------------------------------------------------------------------ the bindings

def test_packed_parameters_are_the_structs():
    r = random.Random(2)
    for pack, struct, floats in ((attn._WEIGHTS_PACK, attn.Kv4WeightsParams, (11,)), (attn._EVICT_PACK, attn.Kv4EvictParams, ())):
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


@pytest.mark.parametrize("call", ["shared", "weights", "evict"])
def test_python_refuses_status_words_of_other_shapes(call):
    ints, x = torch.zeros(4, dtype=torch.int32), torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    f = dict(shared=lambda **kw: kv.kv4_decode_shared(x, None, ints, ints, ints, ints, **kw),
             weights=lambda **kw: kv.kv4_weights(x, None, ints, ints, x, x, **kw),
             evict=lambda **kw: kv.kv4_evict(None, ints, ints, x, keep=1, **kw))[call]
    for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="status"):
            f(status=bad)
    if call == "shared":
        with pytest.raises(ValueError, match="workspace"):
            f(workspace=torch.zeros(1 << 16, dtype=torch.uint8)[::2])


# ------------------------------------------------------------------ the float64 forms

def test_reference_stays_by_hand():
    w = [0.5, 3.0, 1.0, 3.0, float("nan"), 2.0, -1.0, 9.0]
    assert boundedref.stays(w, 4, 1, 1) == [0, 1, 3, 7]
    assert boundedref.stays(w, 3, 0, 1) == [1, 3, 7]
    assert boundedref.stays(w, 2, 0, 0) == [1, 7]
    assert boundedref.stays(w, 3, 5, 5) == [0, 1, 2]
    assert boundedref.stays(w, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]  # NaN goes first
    assert boundedref.stays([1.0] * 6, 4, 1, 1) == [0, 1, 2, 5]   # ties: the lower index


def test_reference_weights_are_the_softmax():
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(1, 16, (4, 1, 16, 64), generator=g)
    scales = torch.rand(4, 1, 16, 2, generator=g, dtype=torch.float64)
    q = torch.randn(1, 2, 3, 64, generator=g, dtype=torch.float64)
    table = [[2, 0, 3]]
    _, lse, _, _ = kvref.decode(q, codes, scales, codes, scales, table, [40], 0.1)
    w = boundedref.weights(q, codes, scales, table, [40], lse, 0.1)[0]
    assert w.shape == (3, 1, 40)
    assert math.isclose(float(w[0].sum()), 6.0, rel_tol=1e-12)  # 2 queries of 3 heads hand out 1 each


def test_reference_eviction_by_hand():
    arrays = [torch.arange(3 * 1 * 4).view(3, 1, 4, 1).to(torch.uint8)]
    w = torch.tensor([[[0.1, 0.9, 0.2, 0.8, 0.3, 0.7, 0.0]]])
    out = w.clone()
    seq, kept = boundedref.evict(arrays, [[2, 0]], [7], w, out, 4, [0], 1)
    assert seq == [4] and kept.tolist() == [[[1, 3, 5, 6]]]
    assert arrays[0].view(-1).tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 9, 11, 1, 2]  # page 2 holds tokens 1 3 | 5 6 of 8..11, 0..2
    assert out[0, 0].tolist()[:4] == pytest.approx([0.9, 0.8, 0.7, 0.0])
    assert boundedref.pages_back([[2, 0]], [7], 4, 4) == [0]
