"""Norm of each query and key head and rotation by position in one pass, with
its gradients (include/gdn2.h, gdn2_rotary_*).

    u = x / sqrt(mean(x^2) + eps) * weight
    (y_a, y_b) = (u_a cos - u_b sin, u_b cos + u_a sin)

over pairs p of values ("halves": p and p + rot / 2, "neighbours": 2 p and
2 p + 1), the angle being positions * inv_freq[p]; rot = 2 * len(inv_freq).
"""
from __future__ import annotations

import ctypes

from . import GDN2_OK, Gdn2Error, _dtype_code, _ptr, load
from ._launch import launch_on, layout_of, no_second_order, want, want_tokens
from .linear import _ref, _scratch

PAIRS = {"halves": 0, "neighbours": 1}


class gdn2_rotary_desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("H_q", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d", ctypes.c_int32),
                ("rot", ctypes.c_int32), ("norm", ctypes.c_int32), ("pairs", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("eps", ctypes.c_float), ("stride_q", ctypes.c_int64),
                ("stride_k", ctypes.c_int64)]


def declare(lib):
    vp, sz, dp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(gdn2_rotary_desc)
    lib.gdn2_rotary_forward.restype, lib.gdn2_rotary_forward.argtypes = ctypes.c_int, [dp] + [vp] * 8 + [vp]
    lib.gdn2_rotary_backward.restype = ctypes.c_int
    lib.gdn2_rotary_backward.argtypes = [dp] + [vp] * 12 + [vp, sz, vp]
    lib.gdn2_rotary_backward_workspace_bytes.restype = sz
    lib.gdn2_rotary_backward_workspace_bytes.argtypes = [dp]


# ------------------------------------------------------------------ raw C ABI
def gdn2_rotary_forward(desc, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, stream=0) -> int:
    return load().gdn2_rotary_forward(_ref(desc), q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, stream)


def gdn2_rotary_backward_workspace_bytes(desc) -> int:
    return load().gdn2_rotary_backward_workspace_bytes(_ref(desc))


def gdn2_rotary_backward(desc, q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, dq, dk, dq_weight, dk_weight,
                         workspace=0, workspace_bytes=0, stream=0) -> int:
    return load().gdn2_rotary_backward(_ref(desc), q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, dq, dk,
                                       dq_weight, dk_weight, workspace, workspace_bytes, stream)


# ------------------------------------------------------------------ torch conveniences
def _problem(q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs):
    import torch
    if pairs not in PAIRS:
        raise ValueError(f"unknown pairs {pairs}")
    if q.dim() < 3 or (k is not None and k.dim() != q.dim()):
        raise ValueError("q and k must be [..., heads, d] with at least one token axis")
    dev, dtype, (*lead, H, d) = q.device, _dtype_code(q), q.shape
    sq = want_tokens(q, "q", q.shape, q.dtype, dev)
    Hk = sk = 0
    if k is not None:
        Hk = k.shape[-2]
        sk = want_tokens(k, "k", (*lead, Hk, d), q.dtype, dev)
    if inv_freq is None or positions is None:
        raise ValueError("positions and inv_freq are required")
    want(inv_freq, "inv_freq", (inv_freq.numel(),), torch.float32, dev)
    want(positions, "positions", torch.Size(lead), torch.int32, dev)
    w = q_weight if q_weight is not None else k_weight
    wdt = q.dtype if w is None else w.dtype
    want(q_weight, "q_weight", (d,), wdt, dev)
    want(k_weight, "k_weight", (d,), wdt, dev)
    if k is None and k_weight is not None:
        raise ValueError("k_weight without k")
    return gdn2_rotary_desc(positions.numel(), H, Hk, d, 2 * inv_freq.numel(), bool(norm), PAIRS[pairs], dtype,
                            dtype if w is None else _dtype_code(w), eps, sq, sk), dev


def _forward(q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs, q_out, k_out, stream):
    import torch
    desc, dev = _problem(q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs)
    want(q_out, "q_out", q.shape, q.dtype, dev)
    if k is not None:
        want(k_out, "k_out", k.shape, q.dtype, dev)
    with launch_on(dev, stream) as handle:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if k_out is None and k is not None:
            k_out = torch.empty(k.shape, dtype=q.dtype, device=dev)
        st = gdn2_rotary_forward(desc, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(positions), _ptr(inv_freq),
                                 _ptr(q_out), _ptr(k_out) if k is not None else None, handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)
    return desc, q_out, k_out if k is not None else None


def rotary_forward(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                   pairs: str = "halves", q_out=None, k_out=None, stream=None):
    """q [..., H_q, d], k [..., H_k, d] or None (bf16 or fp32; views whose
    tokens lie apart, as of a fused projection, are taken as they are),
    positions [...] int32, inv_freq [rot / 2] fp32, weights [d] of one type or
    None. Returns (q_out, k_out), contiguous."""
    return _forward(q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs, q_out, k_out, stream)[1:]


def rotary_backward(q, k, positions, inv_freq, q_weight, k_weight, dq_out, dk_out, eps: float = 1e-6, norm: bool = True,
                    pairs: str = "halves", want_weights: bool = True, grads=None, workspace=None, stream=None) -> dict:
    """Gradients of rotary_forward: a dict with dq, dk (contiguous), dq_weight,
    dk_weight, None where the input is None or it is not wanted. `grads` may
    hold preallocated outputs."""
    import torch
    desc, dev = _problem(q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs)
    for nm, t, like in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if like is not None:
            if t is None:
                raise ValueError(f"{nm} is required")
            want(t, nm, like.shape, q.dtype, dev)
    like = {"dq": q, "dk": k, "dq_weight": q_weight if want_weights else None, "dk_weight": k_weight if want_weights else None}
    g = {nm: None if t is None else (grads or {}).get(nm) for nm, t in like.items()}
    with launch_on(dev, stream) as handle:
        for nm, t in like.items():
            if t is None:
                continue
            if g[nm] is None:
                g[nm] = torch.empty(t.shape, dtype=t.dtype, device=dev)
            else:
                want(g[nm], nm, t.shape, t.dtype, dev)
        _launch_backward(desc, q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out if k is not None else None,
                         g.values(), workspace, handle)
    return g


def _launch_backward(desc, q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, g, workspace, handle):
    """A checked problem, on its device and stream; g: dq, dk, dq_weight, dk_weight."""
    dq, dk, dqw, dkw = g
    need = gdn2_rotary_backward_workspace_bytes(desc) if dqw is not None or dkw is not None else 0
    work = _scratch(workspace, need, q.device)
    st = gdn2_rotary_backward(desc, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(positions), _ptr(inv_freq),
                              _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), _ptr(work),
                              work.numel() if work is not None else 0, handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)


# ------------------------------------------------------------------ autograd
_FN = None


def _autograd_function():
    import torch

    class Rotary(torch.autograd.Function):
        """rotary_forward; saves its inputs (the statistics and angles are
        computed again)."""

        @staticmethod
        def forward(ctx, q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs):
            ctx.desc, qo, ko = _forward(q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs, None, None, None)
            ctx.layout, ctx.problem = layout_of(q, k, positions, inv_freq, q_weight, k_weight), (eps, norm, pairs)
            ctx.save_for_backward(q, k, positions, inv_freq, q_weight, k_weight)
            return qo, ko

        @staticmethod
        def backward(ctx, gq, gk):
            # autograd has made the forward's device and stream current
            no_second_order("rotary")
            q, k, positions, inv_freq, qw, kw = ctx.saved_tensors
            desc = ctx.desc
            if layout_of(q, k, positions, inv_freq, qw, kw) != ctx.layout:  # hooks on saved tensors
                desc, _ = _problem(q, k, positions, inv_freq, qw, kw, *ctx.problem)
            new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
            dq, dk = new(q), None if k is None else new(k)
            dqw = new(qw) if ctx.needs_input_grad[4] else None
            dkw = new(kw) if ctx.needs_input_grad[5] else None
            _launch_backward(desc, q, k, qw, kw, positions, inv_freq, gq.contiguous(),
                             None if k is None else gk.contiguous(), (dq, dk, dqw, dkw), None,
                             torch._C._cuda_getCurrentRawStream(q.device.index))
            return dq, dk, None, None, dqw, dkw, None, None, None

    return Rotary


def rotary(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
           pairs: str = "halves"):
    """Differentiable rotary_forward; gradients reach q, k and the weights."""
    global _FN
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(q, k, positions, inv_freq, q_weight, k_weight, eps, norm, pairs)
