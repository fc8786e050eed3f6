"""Layer norm and root-mean-square norm over the last axis, optionally times
silu(gate), with their gradients (include/gdn2.h, gdn2_norm_*).

    y = (c / sqrt(mean(c^2) + eps) * weight + bias) * silu(gate),
    c = x - mean(x) for kind "layer", x for kind "rms"
"""
from __future__ import annotations

import ctypes

from . import GDN2_OK, Gdn2Error, _dtype_code, _ptr, load
from ._launch import launch_on, want
from .linear import _ref, _scratch

NORM_KINDS = {"layer": 0, "rms": 1}


class gdn2_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int32), ("kind", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("eps", ctypes.c_float)]


def declare(lib):
    vp, sz, dp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(gdn2_norm_desc)
    lib.gdn2_norm_forward.restype, lib.gdn2_norm_forward.argtypes = ctypes.c_int, [dp] + [vp] * 5 + [vp]
    lib.gdn2_norm_backward.restype = ctypes.c_int
    lib.gdn2_norm_backward.argtypes = [dp] + [vp] * 9 + [vp, sz, vp]
    lib.gdn2_norm_backward_workspace_bytes.restype = sz
    lib.gdn2_norm_backward_workspace_bytes.argtypes = [dp]


# ------------------------------------------------------------------ raw C ABI
def gdn2_norm_forward(desc, x, weight, bias, gate, y, stream=0) -> int:
    return load().gdn2_norm_forward(_ref(desc), x, weight, bias, gate, y, stream)


def gdn2_norm_backward_workspace_bytes(desc) -> int:
    return load().gdn2_norm_backward_workspace_bytes(_ref(desc))


def gdn2_norm_backward(desc, x, weight, bias, gate, dy, dx, dweight, dbias, dgate, workspace=0, workspace_bytes=0,
                       stream=0) -> int:
    return load().gdn2_norm_backward(_ref(desc), x, weight, bias, gate, dy, dx, dweight, dbias, dgate, workspace,
                                     workspace_bytes, stream)


# ------------------------------------------------------------------ torch conveniences
def _problem(x, weight, bias, gate, eps, kind):
    if kind not in NORM_KINDS:
        raise ValueError(f"unknown norm {kind}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must be [..., D] with D >= 1, got {tuple(x.shape)}")
    dev, dtype, D = x.device, _dtype_code(x), x.shape[-1]
    w = weight if weight is not None else bias
    wdt = x.dtype if w is None else w.dtype
    want(x, "x", x.shape, x.dtype, dev)
    want(weight, "weight", (D,), wdt, dev)
    want(bias, "bias", (D,), wdt, dev)
    want(gate, "gate", x.shape, x.dtype, dev)
    return gdn2_norm_desc(x.numel() // D, D, NORM_KINDS[kind], dtype, dtype if w is None else _dtype_code(w), eps), dev


def norm_forward(x, weight=None, bias=None, gate=None, eps: float = 1e-5, kind: str = "layer", y=None, stream=None):
    """x, gate [..., D] (bf16 or fp32); weight, bias [D] of one type (bf16 or
    fp32) or None. Returns y like x."""
    import torch
    desc, dev = _problem(x, weight, bias, gate, eps, kind)
    with launch_on(dev, stream) as handle:
        if y is None:
            y = torch.empty_like(x)
        else:
            want(y, "y", x.shape, x.dtype, dev)
        st = gdn2_norm_forward(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), _ptr(y), handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)
    return y


def norm_backward(x, weight, bias, gate, dy, eps: float = 1e-5, kind: str = "layer", want_params: bool = True,
                  want_dgate: bool = True, grads=None, workspace=None, stream=None) -> dict:
    """Gradients of norm_forward: a dict with dx, dgate (like x) and dweight,
    dbias (like weight, bias), None where the input is None or it is not
    wanted. `grads` may hold preallocated outputs."""
    import torch
    desc, dev = _problem(x, weight, bias, gate, eps, kind)
    want(dy, "dy", x.shape, x.dtype, dev)
    if dy is None:
        raise ValueError("dy is required")
    like = {"dx": x, "dweight": weight if want_params else None, "dbias": bias if want_params else None,
            "dgate": gate if want_dgate else None}
    g = {nm: None if t is None else (grads or {}).get(nm) for nm, t in like.items()}
    with launch_on(dev, stream) as handle:
        for nm, t in like.items():
            if t is None:
                continue
            if g[nm] is None:
                g[nm] = torch.empty_like(t)
            else:
                want(g[nm], nm, t.shape, t.dtype, dev)
        work = _scratch(workspace, gdn2_norm_backward_workspace_bytes(desc), dev)
        st = gdn2_norm_backward(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), _ptr(dy), _ptr(g["dx"]),
                                _ptr(g["dweight"]), _ptr(g["dbias"]), _ptr(g["dgate"]), _ptr(work),
                                work.numel() if work is not None else 0, handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)
    return g


# ------------------------------------------------------------------ autograd
_FN = None


def _autograd_function():
    import torch
    from torch.autograd.function import once_differentiable

    class GatedNorm(torch.autograd.Function):
        """norm_forward; saves its inputs (the statistics are computed again)."""

        @staticmethod
        def forward(ctx, x, weight, bias, gate, eps, kind):
            y = norm_forward(x, weight, bias, gate, eps=eps, kind=kind)
            ctx.save_for_backward(x, weight, bias, gate)
            ctx.eps, ctx.kind = eps, kind
            return y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            x, weight, bias, gate = ctx.saved_tensors
            g = norm_backward(x, weight, bias, gate, dy.contiguous(), eps=ctx.eps, kind=ctx.kind,
                              want_params=ctx.needs_input_grad[1] or ctx.needs_input_grad[2],
                              want_dgate=ctx.needs_input_grad[3])
            return g["dx"], g["dweight"], g["dbias"], g["dgate"], None, None

    return GatedNorm


def norm(x, weight=None, bias=None, gate=None, eps: float = 1e-5, kind: str = "layer"):
    """Differentiable norm_forward; gradients reach x, weight, bias and gate."""
    global _FN
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(x, weight, bias, gate, eps, kind)
