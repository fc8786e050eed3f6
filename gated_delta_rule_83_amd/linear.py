"""Gated linear recurrence h_t = a_t * h_{t-1} + b_t * x_t, channel by channel
(include/gdn2.h, gdn2_linear_*): whole and packed sequences, single tokens,
gradients, and the autograd functions.

Gate forms (`gates`): "channel" (a, b fp32), "preact" (a_pre, b_pre in the
input dtype: a = exp(-softplus(a_pre)), b = sigmoid(b_pre)), "tied" (b = 1 - a,
a fp32, b None), "tied_preact" (b = 1 - a, a from its pre-activation, b None).

Everything runs on the tensors' device, on `stream` or its current stream;
tensors that a call makes belong to that stream.
"""
from __future__ import annotations

import ctypes

from . import GDN2_OK, Gdn2Error, _dtype_code, _ptr, load
from ._launch import launch_on, no_second_order, want

LINEAR_CHECKPOINT = 64
LINEAR_GATES = {"channel": 0, "preact": 1, "tied": 2, "tied_preact": 3}


class gdn2_linear_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("gates", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


def declare(lib):
    vp, sz, dp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(gdn2_linear_desc)
    for nm in ("forward", "forward_varlen", "backward", "backward_varlen"):
        f = getattr(lib, f"gdn2_linear_{nm}_workspace_bytes")
        f.restype, f.argtypes = sz, [dp]
    for nm, n in (("forward", 7), ("forward_varlen", 8), ("backward", 11), ("backward_varlen", 12)):
        f = getattr(lib, f"gdn2_linear_{nm}")
        f.restype, f.argtypes = ctypes.c_int, [dp] + [vp] * n + [vp, sz, vp]
    lib.gdn2_linear_step.restype = ctypes.c_int
    lib.gdn2_linear_step.argtypes = [dp] + [vp] * 6 + [vp]


# ------------------------------------------------------------------ raw C ABI
def _ref(desc):
    return None if desc is None else ctypes.byref(desc)


def gdn2_linear_forward_workspace_bytes(desc) -> int:
    return load().gdn2_linear_forward_workspace_bytes(_ref(desc))


def gdn2_linear_forward_varlen_workspace_bytes(desc) -> int:
    return load().gdn2_linear_forward_varlen_workspace_bytes(_ref(desc))


def gdn2_linear_backward_workspace_bytes(desc) -> int:
    return load().gdn2_linear_backward_workspace_bytes(_ref(desc))


def gdn2_linear_backward_varlen_workspace_bytes(desc) -> int:
    return load().gdn2_linear_backward_varlen_workspace_bytes(_ref(desc))


def gdn2_linear_forward(desc, x, a, b, h0, o, h_T, ck, workspace=0, workspace_bytes=0, stream=0) -> int:
    return load().gdn2_linear_forward(_ref(desc), x, a, b, h0, o, h_T, ck, workspace, workspace_bytes, stream)


def gdn2_linear_forward_varlen(desc, cu_seqlens, x, a, b, h0, o, h_T, ck, workspace=0, workspace_bytes=0,
                               stream=0) -> int:
    return load().gdn2_linear_forward_varlen(_ref(desc), cu_seqlens, x, a, b, h0, o, h_T, ck, workspace,
                                             workspace_bytes, stream)


def gdn2_linear_step(desc, x, a, b, h, h_out, o, stream=0) -> int:
    return load().gdn2_linear_step(_ref(desc), x, a, b, h, h_out, o, stream)


def gdn2_linear_backward(desc, x, a, b, h0, ck, dO, dh_T, dx, da, db, dh0, workspace=0, workspace_bytes=0,
                         stream=0) -> int:
    return load().gdn2_linear_backward(_ref(desc), x, a, b, h0, ck, dO, dh_T, dx, da, db, dh0, workspace,
                                       workspace_bytes, stream)


def gdn2_linear_backward_varlen(desc, cu_seqlens, x, a, b, h0, ck, dO, dh_T, dx, da, db, dh0, workspace=0,
                                workspace_bytes=0, stream=0) -> int:
    return load().gdn2_linear_backward_varlen(_ref(desc), cu_seqlens, x, a, b, h0, ck, dO, dh_T, dx, da, db, dh0,
                                              workspace, workspace_bytes, stream)


# ------------------------------------------------------------------ torch conveniences
def _problem(x, a, b, cu, gates, min_dim):
    """(desc, dev, gate dtype, B, saved-state shape) of a checked problem."""
    import torch
    if gates not in LINEAR_GATES:
        raise ValueError(f"unknown gate form {gates}")
    if x.dim() != min_dim:
        raise ValueError(f"x must be {'[T, D]' if cu is not None else '[B, T, D]'}, got {tuple(x.shape)}")
    dev, dtype = x.device, _dtype_code(x)
    T, D = x.shape[-2:]
    if D < 1:
        raise ValueError("x needs at least one channel")
    gdt = x.dtype if gates in ("preact", "tied_preact") else torch.float32
    want(x, "x", x.shape, x.dtype, dev)
    if a is None:
        raise ValueError("a is required")
    want(a, "a", x.shape, gdt, dev)
    if gates in ("tied", "tied_preact"):
        if b is not None:
            raise ValueError(f"b must be None for gates={gates!r} (it is 1 - a)")
    elif b is None:
        raise ValueError(f"b is required for gates={gates!r}")
    want(b, "b", x.shape, gdt, dev)
    tiles = -(-T // LINEAR_CHECKPOINT)
    if cu is None:
        B, rows = x.shape[0], (x.shape[0], tiles, D)
    else:
        want(cu, "cu_seqlens", (cu.numel(),), torch.int32, dev)
        B, rows = cu.numel() - 1, (tiles, D)
        if B < 0:
            raise ValueError("cu_seqlens needs at least one offset")
    return gdn2_linear_desc(B, T, D, LINEAR_GATES[gates], dtype), dev, gdt, B, rows


def _scratch(workspace, need, dev):
    """The caller's workspace, checked, or one of `need` bytes (None for 0)."""
    import torch
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    want(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    return workspace


def _launch_forward(desc, x, a, b, cu, h0, o, h_T, ck, workspace, handle):
    """A checked problem, on its device and stream."""
    need = (gdn2_linear_forward_workspace_bytes if cu is None else gdn2_linear_forward_varlen_workspace_bytes)(desc)
    work = _scratch(workspace, need, x.device)
    ptrs = (_ptr(x), _ptr(a), _ptr(b), _ptr(h0), _ptr(o), _ptr(h_T), _ptr(ck), _ptr(work),
            work.numel() if work is not None else 0, handle)
    if not (x.numel() or (desc.B and h_T is not None)):
        st = GDN2_OK
    elif cu is None:
        st = gdn2_linear_forward(desc, *ptrs)
    else:
        st = gdn2_linear_forward_varlen(desc, _ptr(cu), *ptrs)
    if st != GDN2_OK:
        raise Gdn2Error(st)


def _forward(x, a, b, cu, h0, o, h_T, ck, want_state, want_checkpoints, workspace, stream, gates):
    import torch
    desc, dev, _, B, rows = _problem(x, a, b, cu, gates, 3 if cu is None else 2)
    D, f32 = desc.D, torch.float32
    want(h0, "h0", (B, D), f32, dev)
    want(o, "o", x.shape, x.dtype, dev)
    want(h_T, "h_T", (B, D), f32, dev)
    want(ck, "ck", rows, f32, dev)
    with launch_on(dev, stream) as handle:
        if o is None:
            o = torch.empty_like(x)
        if h_T is None and want_state:
            h_T = torch.empty((B, D), dtype=f32, device=dev)
        if ck is None and want_checkpoints:
            ck = torch.empty(rows, dtype=f32, device=dev)
        _launch_forward(desc, x, a, b, cu, h0, o, h_T, ck, workspace, handle)
    return desc, o, h_T, ck


def linear_forward(x, a, b=None, h0=None, o=None, h_T=None, ck=None, want_state: bool = True,
                   want_checkpoints: bool = False, workspace=None, stream=None, gates: str = "channel"):
    """h_t = a_t h_{t-1} + b_t x_t over whole sequences. x [B,T,D] (bf16 or
    fp32); a, b [B,T,D] by gate form; h0 [B,D] fp32 or None. Returns
    (o [B,T,D], h_T [B,D] fp32), and with want_checkpoints the states saved for
    the backward, ck [B,ceil(T/64),D] fp32."""
    out = _forward(x, a, b, None, h0, o, h_T, ck, want_state, want_checkpoints, workspace, stream, gates)
    return out[1:] if want_checkpoints else out[1:3]


def linear_forward_varlen(x, a, b, cu_seqlens, h0=None, o=None, h_T=None, ck=None, want_state: bool = True,
                          want_checkpoints: bool = False, workspace=None, stream=None, gates: str = "channel"):
    """linear_forward over N packed sequences: x, a, b [T,D]; cu_seqlens int32
    [N+1] on the device (sequence n = rows cu[n]..cu[n+1]-1; rows outside every
    sequence are not written); h0, h_T [N,D]; ck [ceil(T/64),D]."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    out = _forward(x, a, b, cu_seqlens, h0, o, h_T, ck, want_state, want_checkpoints, workspace, stream, gates)
    return out[1:] if want_checkpoints else out[1:3]


def linear_step(x, a, b, h, h_out=None, o=None, stream=None, gates: str = "channel"):
    """One token: x, a, b [N,D] (or [N,1,D]), h [N,D] fp32, replaced by the new
    state unless h_out ([N,D] fp32) is given. Returns o shaped like x."""
    import torch
    if gates not in LINEAR_GATES:
        raise ValueError(f"unknown gate form {gates}")
    if h.dim() != 2 or h.shape[1] < 1:
        raise ValueError(f"h must be [N, D], got {tuple(h.shape)}")
    N, D = h.shape
    dev, dtype = x.device, _dtype_code(x)
    shape = (N, 1, D) if x.dim() == 3 else (N, D)
    gdt = x.dtype if gates in ("preact", "tied_preact") else torch.float32
    if a is None or (b is None) != (gates in ("tied", "tied_preact")):
        raise ValueError(f"gates={gates!r} takes a and {'no b' if gates.startswith('tied') else 'b'}")
    want(x, "x", shape, x.dtype, dev)
    want(a, "a", shape, gdt, dev)
    want(b, "b", shape, gdt, dev)
    want(h, "h", (N, D), torch.float32, dev)
    if h_out is None:
        h_out = h
    else:
        want(h_out, "h_out", (N, D), torch.float32, dev)
    with launch_on(dev, stream) as handle:
        if o is None:
            o = torch.empty_like(x)
        else:
            want(o, "o", shape, x.dtype, dev)
        st = gdn2_linear_step(gdn2_linear_desc(N, 1, D, LINEAR_GATES[gates], dtype), _ptr(x), _ptr(a), _ptr(b),
                              _ptr(h), _ptr(h_out), _ptr(o), handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)
    return o


def _launch_backward(desc, x, a, b, cu, h0, ck, dO, dh_T, g, workspace, handle):
    """A checked problem, on its device and stream; g: dx, da, db, dh0."""
    need = (gdn2_linear_backward_workspace_bytes if cu is None else gdn2_linear_backward_varlen_workspace_bytes)(desc)
    work = _scratch(workspace, need, x.device)
    ptrs = (_ptr(x), _ptr(a), _ptr(b), _ptr(h0), _ptr(ck), _ptr(dO), _ptr(dh_T), *map(_ptr, g), _ptr(work),
            work.numel() if work is not None else 0, handle)
    st = gdn2_linear_backward(desc, *ptrs) if cu is None else gdn2_linear_backward_varlen(desc, _ptr(cu), *ptrs)
    if st != GDN2_OK:
        raise Gdn2Error(st)


def _backward(x, a, b, cu, h0, dO, dh_T, ck, want_dh0, grads, workspace, stream, gates) -> dict:
    import torch
    desc, dev, gdt, B, rows = _problem(x, a, b, cu, gates, 3 if cu is None else 2)
    D, f32 = desc.D, torch.float32
    for t, nm in ((h0, "h0"), (dh_T, "dh_T")):
        want(t, nm, (B, D), f32, dev)
    if dO is None:
        raise ValueError("dO is required")
    want(dO, "dO", x.shape, x.dtype, dev)
    want(ck, "ck", rows, f32, dev)
    grads = grads or {}
    shapes = {"dx": (x.shape, x.dtype), "da": (a.shape, gdt), "db": None if b is None else (b.shape, gdt),
              "dh0": ((B, D), f32) if want_dh0 else None}
    g = {}
    with launch_on(dev, stream) as handle:
        for nm, like in shapes.items():
            g[nm] = t = None if like is None else grads.get(nm)
            if like is not None and t is None:
                g[nm] = torch.empty(like[0], dtype=like[1], device=dev)
            elif t is not None:
                want(t, nm, *like, dev)
        _launch_backward(desc, x, a, b, cu, h0, ck, dO, dh_T, g.values(), workspace, handle)
    return g


def linear_backward(x, a, b, h0, dO, dh_T=None, ck=None, want_dh0: bool = True, grads=None, workspace=None,
                    stream=None, gates: str = "channel") -> dict:
    """Gradients of linear_forward: inputs as there, dO like o, dh_T like h_T or
    None (zero), ck the states linear_forward saved (None: computed again).
    Returns a dict with dx, da, db (None in the tied forms) and dh0 (None
    without want_dh0); `grads` may hold preallocated outputs."""
    return _backward(x, a, b, None, h0, dO, dh_T, ck, want_dh0, grads, workspace, stream, gates)


def linear_backward_varlen(x, a, b, cu_seqlens, h0, dO, dh_T=None, ck=None, want_dh0: bool = True, grads=None,
                           workspace=None, stream=None, gates: str = "channel") -> dict:
    """Gradients of linear_forward_varlen (rows outside every sequence are zero)."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _backward(x, a, b, cu_seqlens, h0, dO, dh_T, ck, want_dh0, grads, workspace, stream, gates)


# ------------------------------------------------------------------ autograd
_FN = None


def _autograd_function():
    import torch

    class GatedLinearRecurrence(torch.autograd.Function):
        """o, h_T of the recurrence; saves the inputs and one state per 64
        tokens. The forward has checked the tensors and autograd gives
        gradients of its outputs' shapes and types: the backward launches."""

        @staticmethod
        def forward(ctx, x, a, b, cu_seqlens, h0, gates):
            ctx.desc, o, h_T, ck = _forward(x, a, b, cu_seqlens, h0, None, None, None, True, True, None, None, gates)
            ctx.save_for_backward(x, a, b, cu_seqlens, h0, ck)
            ctx.set_materialize_grads(False)
            return o, h_T

        @staticmethod
        def backward(ctx, dO, dh_T):
            # autograd has made the forward's device and stream current
            no_second_order("gated_linear_recurrence")
            x, a, b, cu, h0, ck = ctx.saved_tensors
            empty = torch.empty_like
            dO = torch.zeros_like(x) if dO is None else dO.contiguous()
            dh_T = None if dh_T is None else dh_T.contiguous()
            dx, da = empty(x), empty(a)
            db, dh0 = None if b is None else empty(b), None if h0 is None else empty(h0)
            _launch_backward(ctx.desc, x, a, b, cu, h0, ck, dO, dh_T, (dx, da, db, dh0), None,
                             torch._C._cuda_getCurrentRawStream(x.device.index))
            return dx, da, db, None, dh0, None

    return GatedLinearRecurrence


def gated_linear_recurrence(x, a, b=None, h0=None, gates: str = "channel"):
    """Differentiable linear_forward: returns (o, h_T); gradients reach x, a, b and h0."""
    global _FN
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(x, a, b, None, h0, gates)


def gated_linear_recurrence_varlen(x, a, b, cu_seqlens, h0=None, gates: str = "channel"):
    """Differentiable linear_forward_varlen: returns (o, h_T [N,D])."""
    global _FN
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(x, a, b, cu_seqlens, h0, gates)
