"""Softmax attention with grouped heads (include/gdn2.h, gdn2_attention_*,
gdn2_kv_cache_store): whole and packed sequences with their gradients, one new
token over a paged key-value cache, and that cache's writes.

Query i of T_q stands at place i + T_k - T_q of its keys; causal queries see the
keys up to their place, with window > 0 the last `window` of those. A query that
sees nothing (or scores of -inf alone) gives o = 0 and lse = -inf. `scale`
defaults to 1 / sqrt(d).

q, k and v may be views whose tokens lie apart (parts of a fused projection), as
long as a token's heads are contiguous; results are contiguous.
"""
from __future__ import annotations

import ctypes

from . import GDN2_OK, Gdn2Error, _dtype_code, _ptr, load
from ._launch import launch_on, layout_of, no_second_order, want, want_tokens
from .linear import _ref, _scratch


class gdn2_attention_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T_q", ctypes.c_int32), ("T_k", ctypes.c_int32), ("H", ctypes.c_int32),
                ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("stride_q", ctypes.c_int64),
                ("stride_k", ctypes.c_int64), ("stride_v", ctypes.c_int64)]


class gdn2_attention_decode_desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("P", ctypes.c_int32), ("page", ctypes.c_int32), ("M", ctypes.c_int32), ("window", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class gdn2_kv_cache_desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("T", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("P", ctypes.c_int32), ("page", ctypes.c_int32), ("M", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("stride_k", ctypes.c_int64), ("stride_v", ctypes.c_int64)]


def declare(lib):
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    ap, dp, cp = (ctypes.POINTER(x) for x in (gdn2_attention_desc, gdn2_attention_decode_desc, gdn2_kv_cache_desc))
    for nm, first, n, ws in (("attention_forward", ap, 5, False), ("attention_forward_varlen", ap, 7, False),
                             ("attention_backward", ap, 9, True), ("attention_backward_varlen", ap, 11, True),
                             ("attention_decode", dp, 6, True), ("kv_cache_store", cp, 7, False)):
        f = getattr(lib, f"gdn2_{nm}")
        f.restype, f.argtypes = ctypes.c_int, [first] + [vp] * n + ([vp, sz] if ws else []) + [vp]
        if ws:
            f = getattr(lib, f"gdn2_{nm}_workspace_bytes")
            f.restype, f.argtypes = sz, [first]


# ------------------------------------------------------------------ raw C ABI
def gdn2_attention_forward(desc, q, k, v, o, lse, stream=0) -> int:
    return load().gdn2_attention_forward(_ref(desc), q, k, v, o, lse, stream)


def gdn2_attention_forward_varlen(desc, cu_q, cu_k, q, k, v, o, lse, stream=0) -> int:
    return load().gdn2_attention_forward_varlen(_ref(desc), cu_q, cu_k, q, k, v, o, lse, stream)


def gdn2_attention_backward_workspace_bytes(desc) -> int:
    return load().gdn2_attention_backward_workspace_bytes(_ref(desc))


def gdn2_attention_backward_varlen_workspace_bytes(desc) -> int:
    return load().gdn2_attention_backward_varlen_workspace_bytes(_ref(desc))


def gdn2_attention_backward(desc, q, k, v, o, lse, dO, dq, dk, dv, workspace=0, workspace_bytes=0, stream=0) -> int:
    return load().gdn2_attention_backward(_ref(desc), q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes, stream)


def gdn2_attention_backward_varlen(desc, cu_q, cu_k, q, k, v, o, lse, dO, dq, dk, dv, workspace=0, workspace_bytes=0,
                                   stream=0) -> int:
    return load().gdn2_attention_backward_varlen(_ref(desc), cu_q, cu_k, q, k, v, o, lse, dO, dq, dk, dv, workspace,
                                                 workspace_bytes, stream)


def gdn2_attention_decode_workspace_bytes(desc) -> int:
    return load().gdn2_attention_decode_workspace_bytes(_ref(desc))


def gdn2_attention_decode(desc, q, k_cache, v_cache, pages, lengths, o, workspace=0, workspace_bytes=0, stream=0) -> int:
    return load().gdn2_attention_decode(_ref(desc), q, k_cache, v_cache, pages, lengths, o, workspace, workspace_bytes, stream)


def gdn2_kv_cache_store(desc, cu_seqlens, k, v, pages, lengths, k_cache, v_cache, stream=0) -> int:
    return load().gdn2_kv_cache_store(_ref(desc), cu_seqlens, k, v, pages, lengths, k_cache, v_cache, stream)


# ------------------------------------------------------------------ torch conveniences
def _scale(scale, d):
    return d ** -0.5 if scale is None else scale


def _offsets(cu_q, cu_k):
    if cu_q is None:
        raise ValueError("cu_q is required")
    return cu_q, cu_q if cu_k is None else cu_k


def _problem(q, k, v, cu_q, cu_k, scale, causal, window):
    """(desc, dev, shape of lse) of a checked problem; cu_q None: a batch."""
    import torch
    packed = cu_q is not None
    axes = 3 if packed else 4
    if q.dim() != axes or k.dim() != axes or v.dim() != axes:
        raise ValueError(f"q, k and v must be {'[T, heads, d]' if packed else '[B, T, heads, d]'}, got {tuple(q.shape)}, "
                         f"{tuple(k.shape)} and {tuple(v.shape)}")
    dev, dtype = q.device, _dtype_code(q)
    (*lead, T, H, d), (S, Hkv) = q.shape, k.shape[-3:-1]
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"query heads ({H}) must be a multiple of key heads ({Hkv})")
    sq = want_tokens(q, "q", q.shape, q.dtype, dev)
    sk = want_tokens(k, "k", (*lead, S, Hkv, d), q.dtype, dev)
    sv = want_tokens(v, "v", (*lead, S, Hkv, d), q.dtype, dev)
    if packed:
        B = cu_q.numel() - 1
        if B < 0:
            raise ValueError("cu_q needs at least one offset")
        want(cu_q, "cu_q", (B + 1,), torch.int32, dev)
        want(cu_k, "cu_k", (B + 1,), torch.int32, dev)
    else:
        B = lead[0]
    return gdn2_attention_desc(B, T, S, H, Hkv, d, bool(causal), window, dtype, _scale(scale, d), sq, sk, sv), dev, (*lead, H, T)


def _launch_forward(desc, q, k, v, cu_q, cu_k, o, lse, handle):
    if cu_q is None:
        st = gdn2_attention_forward(desc, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), handle)
    else:
        st = gdn2_attention_forward_varlen(desc, _ptr(cu_q), _ptr(cu_k), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)


def _forward(q, k, v, cu_q, cu_k, scale, causal, window, o, lse, stream):
    import torch
    desc, dev, rows = _problem(q, k, v, cu_q, cu_k, scale, causal, window)
    want(o, "o", q.shape, q.dtype, dev)
    want(lse, "lse", rows, torch.float32, dev)
    with launch_on(dev, stream) as handle:
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if lse is None:
            lse = torch.empty(rows, dtype=torch.float32, device=dev)
        _launch_forward(desc, q, k, v, cu_q, cu_k, o, lse, handle)
    return desc, o, lse


def attention_forward(q, k, v, scale=None, causal: bool = True, window: int = 0, o=None, lse=None, stream=None):
    """q [B, T_q, H, d], k, v [B, T_k, H_kv, d] (bf16 or fp32, d 64 or 128).
    Returns (o like q, lse [B, H, T_q] fp32)."""
    return _forward(q, k, v, None, None, scale, causal, window, o, lse, stream)[1:]


def attention_forward_varlen(q, k, v, cu_q, cu_k=None, scale=None, causal: bool = True, window: int = 0, o=None, lse=None,
                             stream=None):
    """Packed sequences: q [T_q, H, d], k, v [T_k, H_kv, d], offsets cu_q, cu_k
    (int32, B + 1; cu_k defaults to cu_q). Returns (o, lse [H, T_q]); rows
    outside every sequence are not written."""
    return _forward(q, k, v, *_offsets(cu_q, cu_k), scale, causal, window, o, lse, stream)[1:]


def _launch_backward(desc, q, k, v, cu_q, cu_k, o, lse, dO, g, workspace, handle):
    """A checked problem, on its device and stream; g: dq, dk, dv."""
    packed = cu_q is not None
    need = (gdn2_attention_backward_varlen_workspace_bytes if packed else gdn2_attention_backward_workspace_bytes)(desc)
    work = _scratch(workspace, need, q.device)
    ptrs = [_ptr(t) for t in (q, k, v, o, lse, dO, *g, work)] + [work.numel() if work is not None else 0, handle]
    st = (gdn2_attention_backward_varlen(desc, _ptr(cu_q), _ptr(cu_k), *ptrs) if packed
          else gdn2_attention_backward(desc, *ptrs))
    if st != GDN2_OK:
        raise Gdn2Error(st)


def _backward(q, k, v, cu_q, cu_k, o, lse, dO, scale, causal, window, grads, workspace, stream):
    import torch
    desc, dev, rows = _problem(q, k, v, cu_q, cu_k, scale, causal, window)
    for nm, t, shape, dt in (("o", o, q.shape, q.dtype), ("lse", lse, rows, torch.float32), ("dO", dO, q.shape, q.dtype)):
        if t is None:
            raise ValueError(f"{nm} is required")
        want(t, nm, shape, dt, dev)
    g = {}
    with launch_on(dev, stream) as handle:
        for nm, t in (("dq", q), ("dk", k), ("dv", v)):
            g[nm] = (grads or {}).get(nm)
            if g[nm] is None:
                g[nm] = torch.empty(t.shape, dtype=t.dtype, device=dev)
            else:
                want(g[nm], nm, t.shape, t.dtype, dev)
        _launch_backward(desc, q, k, v, cu_q, cu_k, o, lse, dO, tuple(g.values()), workspace, handle)
    return g


def attention_backward(q, k, v, o, lse, dO, scale=None, causal: bool = True, window: int = 0, grads=None, workspace=None,
                       stream=None) -> dict:
    """Gradients of attention_forward from its inputs, results and dO: a dict
    with dq, dk, dv (contiguous). `grads` may hold preallocated outputs."""
    return _backward(q, k, v, None, None, o, lse, dO, scale, causal, window, grads, workspace, stream)


def attention_backward_varlen(q, k, v, o, lse, dO, cu_q, cu_k=None, scale=None, causal: bool = True, window: int = 0,
                              grads=None, workspace=None, stream=None) -> dict:
    """Gradients of attention_forward_varlen; rows of no sequence are zero."""
    return _backward(q, k, v, *_offsets(cu_q, cu_k), o, lse, dO, scale, causal, window, grads, workspace, stream)


def kv_cache_empty(P, H_kv, d, page: int = 64, dtype=None, device=None):
    """(k_cache, v_cache) of P pages: [P, H_kv, page, d], cleared."""
    import torch
    dev = torch.device("cuda") if device is None else device
    dt = torch.bfloat16 if dtype is None else dtype
    return tuple(torch.zeros(P, H_kv, page, d, dtype=dt, device=dev) for _ in range(2))


def _cache(k_cache, v_cache, pages, lengths):
    """(P, H_kv, page, d, N, M, dev) of a checked cache and table."""
    import torch
    if k_cache.dim() != 4 or pages.dim() != 2:
        raise ValueError(f"the cache must be [P, H_kv, page, d] and pages [N, M], got {tuple(k_cache.shape)} and {tuple(pages.shape)}")
    dev = k_cache.device
    want(k_cache, "k_cache", k_cache.shape, k_cache.dtype, dev)
    want(v_cache, "v_cache", k_cache.shape, k_cache.dtype, dev)
    want(pages, "pages", pages.shape, torch.int32, dev)
    want(lengths, "lengths", pages.shape[:1], torch.int32, dev)
    return (*k_cache.shape, *pages.shape, dev)


def kv_cache_store(k, v, pages, lengths, k_cache, v_cache, cu_seqlens=None, stream=None):
    """New tokens into the cache: k, v [N, 1, H_kv, d], one token a sequence, or
    with cu_seqlens (int32, N + 1) packed [T, H_kv, d]. lengths [N] int32 count
    the sequences' tokens with the new ones, which are their last; pages [N, M]
    int32. Tokens without a place are skipped; no two tokens of a call may have
    the same one."""
    import torch
    P, Hkv, page, d, N, M, dev = _cache(k_cache, v_cache, pages, lengths)
    dt = k_cache.dtype
    if cu_seqlens is None:
        shape = (N, 1, Hkv, d)
    else:
        want(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
        shape = (k.shape[0], Hkv, d)
    sk, sv = want_tokens(k, "k", shape, dt, dev), want_tokens(v, "v", shape, dt, dev)
    desc = gdn2_kv_cache_desc(N, shape[0], Hkv, d, P, page, M, _dtype_code(k_cache), sk, sv)
    with launch_on(dev, stream) as handle:
        st = gdn2_kv_cache_store(desc, _ptr(cu_seqlens), _ptr(k), _ptr(v), _ptr(pages), _ptr(lengths), _ptr(k_cache),
                                 _ptr(v_cache), handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)


def attention_decode(q, k_cache, v_cache, pages, lengths, scale=None, window: int = 0, o=None, workspace=None, stream=None):
    """One new token a sequence, q [N, 1, H, d], over the first lengths[n] tokens
    of its pages (the new one among them). Returns o like q."""
    import torch
    P, Hkv, page, d, N, M, dev = _cache(k_cache, v_cache, pages, lengths)
    H = q.shape[-2]
    want(q, "q", (N, 1, H, d), k_cache.dtype, dev)
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"query heads ({H}) must be a multiple of key heads ({Hkv})")
    want(o, "o", q.shape, q.dtype, dev)
    desc = gdn2_attention_decode_desc(N, H, Hkv, d, P, page, M, window, _dtype_code(q), _scale(scale, d))
    with launch_on(dev, stream) as handle:
        if o is None:
            o = torch.empty_like(q)
        work = _scratch(workspace, gdn2_attention_decode_workspace_bytes(desc), dev)
        st = gdn2_attention_decode(desc, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(pages), _ptr(lengths), _ptr(o),
                                   _ptr(work), work.numel() if work is not None else 0, handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)
    return o


# ------------------------------------------------------------------ autograd
_FN = None


def _autograd_function():
    import torch

    class Attention(torch.autograd.Function):
        """The forward call; saves its inputs, o and lse."""

        @staticmethod
        def forward(ctx, q, k, v, cu_q, cu_k, scale, causal, window):
            ctx.desc, o, lse = _forward(q, k, v, cu_q, cu_k, scale, causal, window, None, None, None)
            ctx.layout, ctx.problem = layout_of(q, k, v, cu_q, cu_k, o, lse), (scale, causal, window)
            ctx.save_for_backward(q, k, v, cu_q, cu_k, o, lse)
            return o

        @staticmethod
        def backward(ctx, dO):
            # autograd has made the forward's device and stream current
            no_second_order("attention")
            q, k, v, cu_q, cu_k, o, lse = ctx.saved_tensors
            desc = ctx.desc
            if layout_of(q, k, v, cu_q, cu_k, o, lse) != ctx.layout:  # hooks on saved tensors
                desc, dev, rows = _problem(q, k, v, cu_q, cu_k, *ctx.problem)
                want(o, "o", q.shape, q.dtype, dev)
                want(lse, "lse", rows, torch.float32, dev)
            g = tuple(torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
            _launch_backward(desc, q, k, v, cu_q, cu_k, o, lse, dO.contiguous(), g, None,
                             torch._C._cuda_getCurrentRawStream(q.device.index))
            return (*g, None, None, None, None, None)

    return Attention


def _apply(*args):
    global _FN
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(*args)


def attention(q, k, v, scale=None, causal: bool = True, window: int = 0):
    """Differentiable attention_forward (o alone); gradients reach q, k and v."""
    return _apply(q, k, v, None, None, scale, causal, window)


def attention_varlen(q, k, v, cu_q, cu_k=None, scale=None, causal: bool = True, window: int = 0):
    """Differentiable attention_forward_varlen (o alone)."""
    return _apply(q, k, v, *_offsets(cu_q, cu_k), scale, causal, window)
