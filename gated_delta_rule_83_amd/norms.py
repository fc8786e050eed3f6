"""Layer norm and root-mean-square norm over the last axis, optionally times
silu(gate), with their gradients (include/gdn2.h, gdn2_norm_*).

    y = (c / sqrt(mean(c^2) + eps) * weight + bias) * silu(gate),
    c = x - mean(x) for kind "layer", x for kind "rms"
"""
from __future__ import annotations

import ctypes

from . import GDN2_OK, Gdn2Error, _dtype_code, _ptr, load
from ._launch import launch_on, no_second_order, want
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


def _forward(x, weight, bias, gate, eps, kind, y, stream):
    import torch
    desc, dev = _problem(x, weight, bias, gate, eps, kind)
    want(y, "y", x.shape, x.dtype, dev)
    with launch_on(dev, stream) as handle:
        if y is None:
            y = torch.empty_like(x)
        st = gdn2_norm_forward(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), _ptr(y), handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)
    return desc, y


def norm_forward(x, weight=None, bias=None, gate=None, eps: float = 1e-5, kind: str = "layer", y=None, stream=None):
    """x, gate [..., D] (bf16 or fp32); weight, bias [D] of one type (bf16 or
    fp32) or None. Returns y like x."""
    return _forward(x, weight, bias, gate, eps, kind, y, stream)[1]


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
        _launch_backward(desc, x, weight, bias, gate, dy, g.values(), workspace, handle)
    return g


def _launch_backward(desc, x, weight, bias, gate, dy, g, workspace, handle):
    """A checked problem, on its device and stream; g: dx, dweight, dbias, dgate."""
    dx, dw, db, dz = g
    need = gdn2_norm_backward_workspace_bytes(desc) if dw is not None or db is not None else 0
    work = _scratch(workspace, need, x.device)
    st = gdn2_norm_backward(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), _ptr(dy), _ptr(dx), _ptr(dw), _ptr(db),
                            _ptr(dz), _ptr(work), work.numel() if work is not None else 0, handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)


# ------------------------------------------------------------------ autograd
_FN = None


def _autograd_function():
    import torch

    class GatedNorm(torch.autograd.Function):
        """norm_forward; saves its inputs (the statistics are computed again).
        The forward has checked the tensors and autograd gives a gradient of y's
        shape and type: the backward launches."""

        @staticmethod
        def forward(ctx, x, weight, bias, gate, eps, kind):
            ctx.desc, y = _forward(x, weight, bias, gate, eps, kind, None, None)
            ctx.save_for_backward(x, weight, bias, gate)
            return y

        @staticmethod
        def backward(ctx, dy):
            # autograd has made the forward's device and stream current
            no_second_order("norm")
            x, weight, bias, gate = ctx.saved_tensors
            _, need_w, need_b, need_g, _, _ = ctx.needs_input_grad
            desc, empty = ctx.desc, torch.empty_like
            dx = empty(x)
            dw, db, dz = empty(weight) if need_w else None, empty(bias) if need_b else None, empty(gate) if need_g else None
            _launch_backward(desc, x, weight, bias, gate, dy.contiguous(), (dx, dw, db, dz), None,
                             torch._C._cuda_getCurrentRawStream(x.device.index))
            return dx, dw, db, dz, None, None

    return GatedNorm


def norm(x, weight=None, bias=None, gate=None, eps: float = 1e-5, kind: str = "layer"):
    """Differentiable norm_forward; gradients reach x, weight, bias and gate."""
    global _FN
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(x, weight, bias, gate, eps, kind)
