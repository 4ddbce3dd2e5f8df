"""ctypes binding of libattn.so (see include/attn.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or a call fails, an
exception is raised.

Tensors:
  dense: q [B, Sq, Hq, dqk], k [B, Sk, Hkv, dqk], v [B, Sk, Hkv, dv] (any
         strides with a contiguous last dimension);
  THD:   q [Tq, Hq, dqk], ... with int32 ``cu_seqlens_q/k`` on the device.
LSE is float32 [B, Hq, Sq] (dense) or [Hq, Tq] (THD), natural log.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libattn.so")

BF16, FP16, FP32 = 0, 1, 2
_STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED",
           3: "ATTN_ERR_ALIGNMENT", 4: "ATTN_ERR_WORKSPACE", 5: "ATTN_ERR_BAD_METADATA",
           6: "ATTN_ERR_TIMEOUT", 7: "ATTN_ERR_CUDA"}
EXPORTED = ["attn_fwd_workspace_size", "attn_bwd_workspace_size", "attn_fwd", "attn_bwd",
            "attn_bwd_preprocess", "attn_bwd_dq", "attn_bwd_dkdv", "attn_bwd_noalloc",
            "attn_lse_merge", "attn_cp_relayout",
            "attn_query_status", "attn_last_error", "attn_last_launch_count",
            "attn_debug_inject", "attn_host_arena_size", "attn_fwd_bwd_host",
            "attn_fwd_bwd_host_stages", "attn_bwd_path",
            "attn_qk_norm_rope", "attn_qk_norm_rope_bwd", "attn_qk_norm_rope_bwd_workspace_size",
            "attn_kv_plan", "attn_kv_write", "attn_kv_read", "attn_kv_decode",
            "attn_kv_decode_workspace_size"]
# attn_fwd_bwd_host_stages stage bits
HOST_UPLOAD, HOST_COMPUTE, HOST_DOWNLOAD, HOST_ALL = 1, 2, 4, 7
# attn_bwd_path results: which backward kernels run (and the stage order)
BWD_RECOMPUTE, BWD_DS, BWD_PDS = 0, 1, 2
# attn_debug_inject kernel bits (test only)
DEBUG_FWD, DEBUG_DQ, DEBUG_DKDV, DEBUG_SCORES = 1, 2, 4, 8


class AttnError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{_STATUS.get(code, code)}: {msg}")
        self.code = code


class Params(ctypes.Structure):
    """Mirror of attn_params_t."""
    _fields_ = [
        ("dtype", ctypes.c_int), ("o_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int),
        ("batch", ctypes.c_int), ("seqlen_q", ctypes.c_int), ("seqlen_k", ctypes.c_int),
        ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("total_q", ctypes.c_int), ("total_k", ctypes.c_int),
        ("heads_q", ctypes.c_int), ("heads_kv", ctypes.c_int),
        ("d_qk", ctypes.c_int), ("d_v", ctypes.c_int),
        ("stride_q", ctypes.c_int64 * 3), ("stride_k", ctypes.c_int64 * 3),
        ("stride_v", ctypes.c_int64 * 3), ("stride_o", ctypes.c_int64 * 3),
        ("stride_do", ctypes.c_int64 * 3), ("stride_dq", ctypes.c_int64 * 3),
        ("stride_dk", ctypes.c_int64 * 3), ("stride_dv", ctypes.c_int64 * 3),
        ("stride_lse", ctypes.c_int64 * 2),
        ("causal", ctypes.c_int), ("bottom_right", ctypes.c_int),
        ("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
        ("softmax_scale", ctypes.c_float),
        ("accumulate", ctypes.c_int),
        ("seqused_q", ctypes.c_void_p), ("seqused_k", ctypes.c_void_p),
        ("bwd_ds", ctypes.c_int),
    ]


class QkParams(ctypes.Structure):
    """Mirror of attn_qk_params_t."""
    _fields_ = [
        ("dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("batch", ctypes.c_int), ("seqlen", ctypes.c_int), ("heads_q", ctypes.c_int),
        ("heads_k", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("norm", ctypes.c_int),
        ("max_pos", ctypes.c_int), ("eps", ctypes.c_float),
        ("stride_q", ctypes.c_int64 * 3), ("stride_k", ctypes.c_int64 * 3),
        ("stride_qo", ctypes.c_int64 * 3), ("stride_ko", ctypes.c_int64 * 3),
        ("stride_dqo", ctypes.c_int64 * 3), ("stride_dko", ctypes.c_int64 * 3),
    ]


class KvPlanParams(ctypes.Structure):
    """Mirror of attn_kv_plan_params_t."""
    _fields_ = [
        ("batch", ctypes.c_int), ("cols", ctypes.c_int), ("page_size", ctypes.c_int),
        ("num_pages", ctypes.c_int), ("rows", ctypes.c_int), ("n_free", ctypes.c_int),
        ("table_stride", ctypes.c_int64),
    ]


class Kv4CacheDesc(ctypes.Structure):
    """Mirror of attn_kv4_cache_t."""
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("heads_kv", ctypes.c_int),
        ("d_qk", ctypes.c_int), ("d_v", ctypes.c_int),
    ]


class Kv4DecodeParams(ctypes.Structure):
    """Mirror of attn_kv4_decode_params_t."""
    _fields_ = [
        ("dtype", ctypes.c_int), ("o_dtype", ctypes.c_int), ("batch", ctypes.c_int),
        ("seqlen_q", ctypes.c_int), ("heads_q", ctypes.c_int),
        ("stride_q", ctypes.c_int64 * 3), ("stride_o", ctypes.c_int64 * 3),
        ("cols", ctypes.c_int), ("table_stride", ctypes.c_int64),
        ("window_left", ctypes.c_int), ("sinks", ctypes.c_int),
        ("softmax_scale", ctypes.c_float),
    ]


_lib = None
_fast = None
_lock = threading.Lock()


def load():
    """Load libattn.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "bwd_tcgen05_tmem_gb300.build.build() (nvcc, sm_103a)")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(Params)
        vp, sz, i64p = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int64)
        lib.attn_fwd_workspace_size.argtypes = [P]
        lib.attn_fwd_workspace_size.restype = sz
        lib.attn_bwd_workspace_size.argtypes = [P]
        lib.attn_bwd_workspace_size.restype = sz
        lib.attn_bwd_path.argtypes = [P]
        lib.attn_bwd_path.restype = ctypes.c_int
        lib.attn_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.attn_fwd.restype = ctypes.c_int
        for name in ("attn_bwd", "attn_bwd_preprocess", "attn_bwd_dq", "attn_bwd_dkdv"):
            fn = getattr(lib, name)
            fn.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            fn.restype = ctypes.c_int
        lib.attn_bwd_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.attn_bwd_noalloc.restype = ctypes.c_int
        lib.attn_lse_merge.argtypes = [ctypes.c_int, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                       i64p, i64p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                       vp, ctypes.c_int, vp, vp]
        lib.attn_lse_merge.restype = ctypes.c_int
        i64p = ctypes.POINTER(ctypes.c_int64)
        lib.attn_cp_relayout.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                         ctypes.c_int, ctypes.c_int, vp, i64p, vp, i64p, vp]
        lib.attn_cp_relayout.restype = ctypes.c_int
        lib.attn_query_status.argtypes = [vp, vp]
        lib.attn_query_status.restype = ctypes.c_int
        lib.attn_last_error.argtypes = []
        lib.attn_last_error.restype = ctypes.c_char_p
        lib.attn_last_launch_count.argtypes = []
        lib.attn_last_launch_count.restype = ctypes.c_int
        lib.attn_debug_inject.argtypes = [ctypes.c_uint, ctypes.c_int, ctypes.c_uint64]
        lib.attn_debug_inject.restype = None
        lib.attn_host_arena_size.argtypes = [P]
        lib.attn_host_arena_size.restype = sz
        lib.attn_fwd_bwd_host.argtypes = [P] + [vp] * 9 + [vp, sz, vp]
        lib.attn_fwd_bwd_host.restype = ctypes.c_int
        lib.attn_fwd_bwd_host_stages.argtypes = [P] + [vp] * 9 + [vp, sz, ctypes.c_uint, vp]
        lib.attn_fwd_bwd_host_stages.restype = ctypes.c_int
        QP = ctypes.POINTER(QkParams)
        lib.attn_qk_norm_rope.argtypes = [QP] + [vp] * 11
        lib.attn_qk_norm_rope.restype = ctypes.c_int
        lib.attn_qk_norm_rope_bwd_workspace_size.argtypes = [QP]
        lib.attn_qk_norm_rope_bwd_workspace_size.restype = sz
        lib.attn_qk_norm_rope_bwd.argtypes = [QP] + [vp] * 14 + [sz, vp, vp]
        lib.attn_qk_norm_rope_bwd.restype = ctypes.c_int
        lib.attn_kv_plan.argtypes = [ctypes.POINTER(KvPlanParams)] + [vp] * 12
        lib.attn_kv_plan.restype = ctypes.c_int
        C = ctypes.POINTER(Kv4CacheDesc)
        for name in ("attn_kv_write", "attn_kv_read"):
            fn = getattr(lib, name)
            fn.argtypes = [C, ctypes.c_int, ctypes.c_int, vp, i64p, vp, i64p, vp, vp, vp]
            fn.restype = ctypes.c_int
        D = ctypes.POINTER(Kv4DecodeParams)
        lib.attn_kv_decode_workspace_size.argtypes = [D, C]
        lib.attn_kv_decode_workspace_size.restype = sz
        lib.attn_kv_decode.argtypes = [D, C] + [vp] * 6 + [sz, vp, vp]
        lib.attn_kv_decode.restype = ctypes.c_int
        global _fast
        _fast = _fast_handle()
        _lib = lib
        return lib


# Calls that a serving step makes for every token take their parameter structs
# as packed bytes, through a second handle of the library: filling a ctypes
# structure field by field costs several microseconds, packing it less than one.
_QK_PACK = struct.Struct("@11if18q").pack          # attn_qk_params_t
_PLAN_PACK = struct.Struct("@6iq").pack            # attn_kv_plan_params_t
_DECODE_PACK = struct.Struct("@5i6qiq2if0q").pack  # attn_kv4_decode_params_t


def _fast_handle():
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    for name, args in (("attn_qk_norm_rope", [vp] * 12),
                       ("attn_qk_norm_rope_bwd", [vp] * 15 + [sz, vp, vp]),
                       ("attn_kv_plan", [vp] * 13),
                       ("attn_kv_write", [vp, ci, ci] + [vp] * 7),
                       ("attn_kv_read", [vp, ci, ci] + [vp] * 7),
                       ("attn_kv_decode", [vp] * 8 + [sz, vp, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    for name, args in (("attn_qk_norm_rope_bwd_workspace_size", [vp]),
                       ("attn_kv_decode_workspace_size", [vp, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, sz
    return lib


def fast():
    if _fast is None:
        load()
    return _fast


def _check(rc):
    if rc != 0:
        msg = load().attn_last_error().decode(errors="replace")
        raise AttnError(rc, msg)


def last_launch_count():
    return load().attn_last_launch_count()


def _code(dt):
    if dt in (torch.bfloat16, "bf16"):
        return BF16
    if dt in (torch.float16, "fp16"):
        return FP16
    if dt in (torch.float32, "fp32"):
        return FP32
    raise ValueError(f"unsupported dtype {dt}")


def _strides(t, thd):
    if t is None:
        return (0, 0, 0)
    if t.stride(-1) != 1:
        raise ValueError("the head-dim axis must be contiguous")
    if thd:
        return (0, t.stride(0), t.stride(1))
    return (t.stride(0), t.stride(1), t.stride(2))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def make_params(q, k, v, *, causal=True, scale=None, window=(-1, -1), bottom_right=False,
                cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None,
                o=None, dout=None, dq=None, dk=None, dv=None, o_dtype=None, grad_dtype=None,
                lse_strides=(0, 0), accumulate=False, seqused_q=None, seqused_k=None,
                bwd_ds=0):
    """attn_params_t for these tensors.  ``bwd_ds``: 0 auto, 1 always, -1
    never keep dS in the backward's workspace (attn_bwd_path)."""
    thd = cu_seqlens_q is not None
    p = Params()
    p.dtype = _code(q.dtype)
    p.o_dtype = _code(o_dtype if o_dtype is not None else (o.dtype if o is not None else q.dtype))
    p.grad_dtype = _code(grad_dtype if grad_dtype is not None else q.dtype)
    if thd:
        if cu_seqlens_k is None:
            cu_seqlens_k = cu_seqlens_q
        p.batch = cu_seqlens_q.numel() - 1
        p.cu_seqlens_q = cu_seqlens_q.data_ptr()
        p.cu_seqlens_k = cu_seqlens_k.data_ptr()
        p.total_q, p.total_k = q.shape[0], k.shape[0]
        p.seqlen_q = int(max_seqlen_q if max_seqlen_q is not None else q.shape[0])
        p.seqlen_k = int(max_seqlen_k if max_seqlen_k is not None else k.shape[0])
        hq, dqk = q.shape[1], q.shape[2]
        hkv, dvd = k.shape[1], v.shape[2]
    else:
        p.batch, p.seqlen_q, hq, dqk = q.shape
        p.seqlen_k, hkv, dvd = k.shape[1], k.shape[2], v.shape[3]
    p.heads_q, p.heads_kv, p.d_qk, p.d_v = hq, hkv, dqk, dvd
    for name, t in (("stride_q", q), ("stride_k", k), ("stride_v", v), ("stride_o", o),
                    ("stride_do", dout), ("stride_dq", dq), ("stride_dk", dk),
                    ("stride_dv", dv)):
        getattr(p, name)[:] = _strides(t, thd)
    p.stride_lse[:] = lse_strides
    p.causal = int(bool(causal))
    p.bottom_right = int(bool(bottom_right))
    p.window_left, p.window_right = int(window[0]), int(window[1])
    p.softmax_scale = float(scale if scale is not None else 1.0 / math.sqrt(dqk))
    p.accumulate = int(bool(accumulate))
    p.bwd_ds = int(bwd_ds)
    if seqused_q is not None:  # padded THD: device int32 [batch] visible lengths
        p.seqused_q = seqused_q.data_ptr()
        p.seqused_k = (seqused_k if seqused_k is not None else seqused_q).data_ptr()
    return p


def _lse_shape(q, thd):
    if thd:
        return (q.shape[1], q.shape[0])
    return (q.shape[0], q.shape[2], q.shape[1])


def fwd(q, k, v, *, causal=True, scale=None, window=(-1, -1), bottom_right=False,
        cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None,
        seqused_q=None, seqused_k=None, out=None, lse=None, o_dtype=None, lse_strides=(0, 0),
        workspace=None, stream=None):
    """Fused attention forward. Returns (o, lse).  lse_strides: element strides
    {batch, head} of `lse` ((0, 0) = its default layout)."""
    lib = load()
    thd = cu_seqlens_q is not None
    odt = o_dtype if o_dtype is not None else (out.dtype if out is not None else q.dtype)
    if out is None:
        shape = (*q.shape[:-2], q.shape[-2], v.shape[-1])
        out = torch.empty(shape, dtype=odt, device=q.device)
    if lse is None:
        lse = torch.empty(_lse_shape(q, thd), dtype=torch.float32, device=q.device)
    p = make_params(q, k, v, causal=causal, scale=scale, window=window,
                    bottom_right=bottom_right, cu_seqlens_q=cu_seqlens_q,
                    cu_seqlens_k=cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                    max_seqlen_k=max_seqlen_k, o=out, o_dtype=odt, lse_strides=lse_strides,
                    seqused_q=seqused_q, seqused_k=seqused_k)
    need = lib.attn_fwd_workspace_size(ctypes.byref(p))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(lib.attn_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                        _ptr(workspace), workspace.numel(), _stream(stream)))
    return out, lse


def bwd(q, k, v, o, dout, lse, *, causal=True, scale=None, window=(-1, -1),
        bottom_right=False, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None,
        max_seqlen_k=None, seqused_q=None, seqused_k=None, dq=None, dk=None, dv=None,
        grad_dtype=None, lse_strides=(0, 0), accumulate=False, workspace=None, stream=None,
        stage="all", bwd_ds=0):
    """Fused attention backward. Returns (dq, dk, dv).

    ``stage``: "all" (attn_bwd), or one of "preprocess", "dq", "dkdv" to run a
    single stage of it (the C ABI's attn_bwd_* entry points; on the BWD_DS
    path the dkdv stage comes before the dq stage).  ``bwd_ds``: see
    make_params."""
    lib = load()
    gdt = grad_dtype if grad_dtype is not None else q.dtype
    if dq is None:
        dq = torch.empty(q.shape, dtype=gdt, device=q.device)
    if dk is None:
        dk = torch.empty(k.shape, dtype=gdt, device=q.device)
    if dv is None:
        dv = torch.empty(v.shape, dtype=gdt, device=q.device)
    p = make_params(q, k, v, causal=causal, scale=scale, window=window,
                    bottom_right=bottom_right, cu_seqlens_q=cu_seqlens_q,
                    cu_seqlens_k=cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                    max_seqlen_k=max_seqlen_k, o=o, dout=dout, dq=dq, dk=dk, dv=dv,
                    o_dtype=o.dtype, grad_dtype=gdt, lse_strides=lse_strides,
                    accumulate=accumulate, seqused_q=seqused_q, seqused_k=seqused_k,
                    bwd_ds=bwd_ds)
    need = lib.attn_bwd_workspace_size(ctypes.byref(p))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    fn = {"all": lib.attn_bwd, "preprocess": lib.attn_bwd_preprocess, "dq": lib.attn_bwd_dq,
          "dkdv": lib.attn_bwd_dkdv}[stage]
    _check(fn(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout),
                        _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                        workspace.numel(), _stream(stream)))
    return dq, dk, dv


def bwd_noalloc(q, k, v, o, dout, lse, *, causal=True, scale=None, window=(-1, -1),
                bottom_right=False, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None,
                max_seqlen_k=None, dq=None, dk=None, dv=None, grad_dtype=None,
                lse_strides=(0, 0), accumulate=False, stream=None):
    """attn_bwd_noalloc: the backward without a caller workspace.

    For callers that must not allocate device memory while they run (the
    library's own 8 MiB static scratch area is used instead; concurrent calls
    on one device race).  The output tensors are still the caller's.
    Returns (dq, dk, dv)."""
    lib = load()
    gdt = grad_dtype if grad_dtype is not None else q.dtype
    if dq is None:
        dq = torch.empty(q.shape, dtype=gdt, device=q.device)
    if dk is None:
        dk = torch.empty(k.shape, dtype=gdt, device=q.device)
    if dv is None:
        dv = torch.empty(v.shape, dtype=gdt, device=q.device)
    p = make_params(q, k, v, causal=causal, scale=scale, window=window,
                    bottom_right=bottom_right, cu_seqlens_q=cu_seqlens_q,
                    cu_seqlens_k=cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                    max_seqlen_k=max_seqlen_k, o=o, dout=dout, dq=dq, dk=dk, dv=dv,
                    o_dtype=o.dtype, grad_dtype=gdt, lse_strides=lse_strides,
                    accumulate=accumulate)
    _check(lib.attn_bwd_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout),
                                _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _stream(stream)))
    return dq, dk, dv


def _host_params(q, k, v, dout, o, dq, dk, dv, kw):
    for name, t in (("q", q), ("k", k), ("v", v), ("dout", dout), ("o", o), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        if t.is_cuda:
            raise ValueError(f"{name} must be a host tensor")
    return make_params(q, k, v, o=o, dout=dout, dq=dq, dk=dk, dv=dv, o_dtype=o.dtype,
                       grad_dtype=dq.dtype, **kw)


def host_arena_size(q, k, v, dout, o, dq, dk, dv, **kw):
    """Bytes of device arena attn_fwd_bwd_host needs for these host tensors."""
    p = _host_params(q, k, v, dout, o, dq, dk, dv, kw)
    return load().attn_host_arena_size(ctypes.byref(p))


def fwd_bwd_host(q, k, v, dout, o, lse, dq, dk, dv, arena, *, stream=None, stages=HOST_ALL,
                 **kw):
    """attn_fwd_bwd_host: one forward + backward step whose inputs (q, k, v,
    dout) and outputs (o, lse, dq, dk, dv) are HOST tensors (pinned for the
    copies to overlap); ``arena`` is a device uint8 tensor of at least
    host_arena_size() bytes.  THD ``cu_seqlens_q/k`` (and ``seqused_q/k``) in
    ``kw`` are host int32 tensors too.  Enqueued on ``stream``; the outputs are
    valid once it has passed the call.  ``stages``: a mask of HOST_UPLOAD,
    HOST_COMPUTE and HOST_DOWNLOAD (attn_fwd_bwd_host_stages) to run part of
    the step, e.g. to pipeline consecutive steps over several streams."""
    lib = load()
    if lse.is_cuda or not arena.is_cuda:
        raise ValueError("lse must be a host tensor and arena a device tensor")
    p = _host_params(q, k, v, dout, o, dq, dk, dv, kw)
    args = (ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(o), _ptr(lse),
            _ptr(dq), _ptr(dk), _ptr(dv), _ptr(arena), arena.numel())
    if stages == HOST_ALL:
        _check(lib.attn_fwd_bwd_host(*args, _stream(stream)))
    else:
        _check(lib.attn_fwd_bwd_host_stages(*args, int(stages), _stream(stream)))
    return o, lse, dq, dk, dv


def bwd_path(q, k, v, **kw):
    """attn_bwd_path: BWD_RECOMPUTE, BWD_DS or BWD_PDS for these tensors."""
    p = make_params(q, k, v, **kw)
    r = load().attn_bwd_path(ctypes.byref(p))
    if r < 0:
        raise AttnError(1, load().attn_last_error().decode(errors="replace"))
    return r


def workspace_size(kind, q, k, v, **kw):
    """Bytes of workspace attn_fwd ('fwd') or attn_bwd ('bwd') needs."""
    p = make_params(q, k, v, **kw)
    fn = load().attn_fwd_workspace_size if kind == "fwd" else load().attn_bwd_workspace_size
    return fn(ctypes.byref(p))


def lse_merge(o_parts, lse_parts, row0, nrows, rows, *, out=None, lse_out=None,
              out_dtype=torch.bfloat16, stream=None):
    """LSE-weighted merge.  o_parts[i]: fp32 [nrows[i], H, dv]; lse_parts[i]: fp32
    [H, nrows[i]]; part i covers output rows [row0[i], row0[i] + nrows[i])."""
    lib = load()
    n = len(o_parts)
    heads, dvd = o_parts[0].shape[1], o_parts[0].shape[2]
    if out is None:
        out = torch.empty((rows, heads, dvd), dtype=out_dtype, device=o_parts[0].device)
    if lse_out is None:
        lse_out = torch.empty((heads, rows), dtype=torch.float32, device=o_parts[0].device)
    optrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in o_parts])
    lptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in lse_parts])
    r0 = (ctypes.c_int64 * n)(*[int(x) for x in row0])
    nr = (ctypes.c_int64 * n)(*[int(x) for x in nrows])
    _check(lib.attn_lse_merge(n, optrs, lptrs, r0, nr, int(rows), int(heads), int(dvd),
                              _ptr(out), _code(out.dtype), _ptr(lse_out), _stream(stream)))
    return out, lse_out


def debug_inject(kernel_mask, drop_load, wait_limit_ns=0):
    """TEST ONLY: arm attn_debug_inject for the next attn_fwd / attn_bwd call on
    this thread (the first CTA of each selected kernel leaves out load
    ``drop_load`` and waits at most ``wait_limit_ns``; 0 keeps 2 s)."""
    load().attn_debug_inject(int(kernel_mask), int(drop_load), int(wait_limit_ns))


def query_status(workspace, stream=None):
    """Synchronise the stream and raise if the device status word is set."""
    _check(load().attn_query_status(_ptr(workspace), _stream(stream)))


def cp_relayout(src, dst, *, to_heads, cp, stream=None):
    """All-to-all CP relayout between sequence shards and head shards.

    Token-major tensors (Q, K, V, O, dO, gradients): sequence side
    [cp, 2*chunk, heads, d], head side [cp, seqlen, heads/cp, d].
    LSE-like FP32 tensors (head-major): sequence side [cp, heads, 2*chunk],
    head side [cp, heads/cp, seqlen].  to_heads: src is the sequence side."""
    seq, head = (src, dst) if to_heads else (dst, src)
    if seq.dim() == 4:  # [cp, tokens, heads, d]
        seqlen, heads, d = head.shape[1], seq.shape[2], seq.shape[3]
        ss = (seq.stride(0), seq.stride(1), seq.stride(2))
        hs = (head.stride(0), head.stride(1), head.stride(2))
        assert seq.stride(3) == 1 and head.stride(3) == 1, "d must be contiguous"
    else:  # [cp, heads, tokens]
        seqlen, heads, d = head.shape[2], seq.shape[1], 1
        ss = (seq.stride(0), seq.stride(2), seq.stride(1))
        hs = (head.stride(0), head.stride(2), head.stride(1))
    assert src.dtype == dst.dtype
    arr = ctypes.c_int64 * 3
    s_src, s_dst = (arr(*ss), arr(*hs)) if to_heads else (arr(*hs), arr(*ss))
    _check(load().attn_cp_relayout(int(bool(to_heads)), cp, seqlen, heads, d, src.element_size(),
                                   _ptr(src), s_src, _ptr(dst), s_dst, _stream(stream)))
    return dst


# ----------------------------------------------------- norm and rotation of q and k

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_CODES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


def on_device(t, *others):
    """The device index of CUDA tensor ``t``, on which ``others`` (None apart) must lie too."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError(f"tensors are on {t.device} and {o.device}")
    return dev


def check_buffers(status, workspace=None):
    """What the kernels write as words and bytes from an address on (None: not given)."""
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status must be an int32 tensor of one element or more")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def launch(dev, stream, fn, *args):
    """fn(*args, stream) with device ``dev`` current; raises on an error status."""
    if stream is not None:
        s = stream.cuda_stream
    elif _raw_stream is not None:
        s = _raw_stream(dev)
    else:
        s = torch.cuda.current_stream(dev).cuda_stream
    if dev == torch.cuda.current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        _check(rc)


def new(shape, dtype, dev, stream):
    """A new tensor for work on ``stream`` (None: the current one): memory of that
    stream, so that it is not handed out again while the work is under way."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _sized(dev, fn, *args):
    """fn(*args) with device ``dev`` current (workspace sizes follow its SM count)."""
    if dev == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _qk_strides(name, t, shape, dtype):
    """{batch, token, head} strides of a tensor that must have this shape and dtype."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, q has {dtype}")
    s = t.stride()
    if s[-1] != 1:
        raise ValueError("the head-dim axis must be contiguous")
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


_NO_STRIDES = (0, 0, 0)


def _qk_pack(q, k, cos, sin, positions, wq, wk, norm, eps, interleaved, qo, ko, dqo, dko):
    shape, dt = q.shape, q.dtype
    if len(shape) == 4:
        b, s, hq, d = shape
    elif len(shape) == 3:
        b = 1
        s, hq, d = shape
    else:
        raise ValueError("q must be [batch, seqlen, heads, d] or [total, heads, d]")
    hk, k_shape = 0, None
    sk = sko = _NO_STRIDES
    if k is not None:
        if k.dim() != len(shape):
            raise ValueError("k must have as many axes as q")
        hk = k.shape[-2]
        k_shape = (*shape[:-2], hk, d)
        sk = _qk_strides("k", k, k_shape, dt)
        sko = _qk_strides("k_out (dk)", ko, k_shape, dt)
    elif ko is not None:
        raise ValueError("an output for k without k")
    rot = max_pos = 0
    if cos is not None and sin is not None:
        if (cos.shape != sin.shape or cos.dim() != 2 or cos.dtype != torch.float32
                or sin.dtype != torch.float32 or not cos.is_contiguous() or not sin.is_contiguous()):
            raise ValueError("cos and sin must be contiguous float32 [max_pos, rotary_dim / 2]")
        max_pos, rot = cos.shape
        rot *= 2
    elif cos is not None or sin is not None:
        raise ValueError("cos and sin must both be given or None")
    if positions is not None and (positions.dtype != torch.int32 or positions.numel() != b * s
                                  or not positions.is_contiguous()):
        raise ValueError("positions must be contiguous int32, one for each token")
    wdt = torch.float32
    if wq is not None or wk is not None:
        wdt = (wq if wq is not None else wk).dtype
        for w in (wq, wk):
            if w is not None and (w.shape != (d,) or w.dtype != wdt or not w.is_contiguous()):
                raise ValueError("norm weights must be contiguous [head_dim] and of one dtype")
    sdq = _qk_strides("dq_out", dqo, shape, dt) if dqo is not None else _NO_STRIDES
    sdk = _qk_strides("dk_out", dko, k_shape, dt) if dko is not None else _NO_STRIDES
    if dt not in _CODES or wdt not in _CODES:
        raise ValueError(f"unsupported dtypes {dt}, {wdt}")
    return _QK_PACK(_CODES[dt], _CODES[wdt], b, s, hq, hk, d, rot, bool(interleaved), bool(norm),
                    max_pos, eps, *_qk_strides("q", q, shape, dt), *sk,
                    *_qk_strides("q_out (dq)", qo, shape, dt), *sko, *sdq, *sdk)


def qk_norm_rope(q, k, cos, sin, *, positions=None, wq=None, wk=None, norm=True, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, status=None, stream=None):
    """Norm of each query and key head and rotation by its position, in one
    pass (attn_qk_norm_rope).  Returns (q_out, k_out).

    q [B, S, Hq, d] or [T, Hq, d]; k likewise or None; cos, sin: float32
    [max_pos, rotary_dim / 2], or None for no rotation; positions: int32 [B, S]
    or [T], negative for padding rows (left as they are in ``q_out`` and
    ``k_out``), or None for 0, 1, ...; wq, wk: [d] or None.  ``q_out=q`` works
    in place.  ``status``: int32 device word (see include/attn.h), or None."""
    check_buffers(status)
    lib = fast()
    dev = on_device(q, k, cos, sin, positions, wq, wk, q_out, k_out, status)
    if q_out is None:
        q_out = new(q.shape, q.dtype, dev, stream)
    if k_out is None and k is not None:
        k_out = new(k.shape, q.dtype, dev, stream)
    p = _qk_pack(q, k, cos, sin, positions, wq, wk, norm, eps, interleaved, q_out, k_out, None,
                 None)
    launch(dev, stream, lib.attn_qk_norm_rope, p, q.data_ptr(),
           None if k is None else k.data_ptr(), None if wq is None else wq.data_ptr(),
           None if wk is None else wk.data_ptr(), None if cos is None else cos.data_ptr(),
           None if sin is None else sin.data_ptr(),
           None if positions is None else positions.data_ptr(), q_out.data_ptr(),
           None if k_out is None else k_out.data_ptr(),
           None if status is None else status.data_ptr())
    return q_out, k_out


def qk_norm_rope_bwd(q, k, cos, sin, dq_out, dk_out, *, positions=None, wq=None, wk=None,
                     norm=True, eps=1e-6, interleaved=False, dq=None, dk=None, dwq=None,
                     dwk=None, workspace=None, status=None, stream=None):
    """Gradient of qk_norm_rope: (dq, dk, dwq, dwk) from its inputs q, k and the
    gradients of its outputs.  dwq and dwk are float32 [d] (None without
    weights); rows of padding tokens are left as they are in dq and dk."""
    check_buffers(status, workspace)
    lib = fast()
    dev = on_device(q, k, cos, sin, dq_out, dk_out, positions, wq, wk, dq, dk, dwq, dwk,
                    workspace, status)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out must both be given or None")
    d = q.shape[-1]
    if dq is None:
        dq = new(q.shape, q.dtype, dev, stream)
    if dk is None and k is not None:
        dk = new(k.shape, q.dtype, dev, stream)
    if wq is not None and dwq is None:
        dwq = new((d,), torch.float32, dev, stream)
    if wk is not None and dwk is None and k is not None:
        dwk = new((d,), torch.float32, dev, stream)
    for w in (dwq, dwk):
        if w is not None and (w.dtype != torch.float32 or w.shape != (d,) or not w.is_contiguous()):
            raise ValueError("weight gradients must be contiguous float32 [head_dim]")
    p = _qk_pack(q, k, cos, sin, positions, wq, wk, norm, eps, interleaved, dq, dk, dq_out,
                 dk_out)
    if workspace is None:
        workspace = new((_sized(dev, lib.attn_qk_norm_rope_bwd_workspace_size, p),), torch.uint8,
                        dev, stream)
    launch(dev, stream, lib.attn_qk_norm_rope_bwd, p, q.data_ptr(),
           None if k is None else k.data_ptr(), None if wq is None else wq.data_ptr(),
           None if wk is None else wk.data_ptr(), None if cos is None else cos.data_ptr(),
           None if sin is None else sin.data_ptr(),
           None if positions is None else positions.data_ptr(), dq_out.data_ptr(),
           None if dk_out is None else dk_out.data_ptr(), dq.data_ptr(),
           None if dk is None else dk.data_ptr(), None if dwq is None else dwq.data_ptr(),
           None if dwk is None else dwk.data_ptr(), workspace.data_ptr(), workspace.nbytes,
           None if status is None else status.data_ptr())
    return dq, dk, dwq, dwk


def rope_tables(max_pos, rotary_dim, *, base=10000.0, device="cuda"):
    """cos, sin (float32 [max_pos, rotary_dim / 2]) of the angles pos *
    base^(-2 i / rotary_dim), computed in float64: an angle of 10^6 has an
    error of 0.03 in float32."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    ang = (torch.arange(max_pos, dtype=torch.float64, device=device)[:, None]
           * base ** (-2.0 * i / rotary_dim))
    return ang.cos().float(), ang.sin().float()
