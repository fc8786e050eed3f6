"""Plain 64-bit forms of the linear recurrence, the norms and the 8-bit state
cache, and error bounds for them (test infrastructure, numpy only).

U32 is one rounding to fp32 (half a step, relative); half(t) the same for a
tensor's type."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
FORMS = ("channel", "preact", "tied", "tied_preact")


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def gates_of(a, b, form):
    """(decay, input gate) in 64 bits."""
    if form == "preact":
        return sigmoid(-a), sigmoid(b)
    if form == "tied_preact":
        return sigmoid(-a), sigmoid(a)
    return (a, 1.0 - a) if form == "tied" else (a, b)


def linear(x, a, b, h0, form):
    """Token by token over [T, D]: (o, h_T)."""
    A, Bg = gates_of(a, b, form)
    h, o = h0.copy(), np.empty_like(x)
    for t in range(x.shape[0]):
        h = A[t] * h + Bg[t] * x[t]
        o[t] = h
    return o, h


def linear_grads(x, a, b, h0, dO, dhT, form):
    """dx, da, db (None in the tied forms), dh0, and the adjoints g [T, D]."""
    A, Bg = gates_of(a, b, form)
    o, _ = linear(x, a, b, h0, form)
    m, T = dhT.copy(), x.shape[0]
    dx, da, db, g = (np.empty_like(x) for _ in range(4))
    for t in reversed(range(T)):
        g[t] = dO[t] + m
        dx[t], db[t], da[t] = Bg[t] * g[t], x[t] * g[t], (o[t - 1] if t else h0) * g[t]
        m = A[t] * g[t]
    if form in ("tied", "tied_preact"):
        da, db = da - db, None
    if form in ("preact", "tied_preact"):
        da = -da * A * sigmoid(a)
        db = None if db is None else db * Bg * sigmoid(-b)
    return dx, da, db, m, g


def norm(x, w, b, z, eps, kind):
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    xh = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = xh * (1.0 if w is None else w) + (0.0 if b is None else b)
    return n if z is None else n * z * sigmoid(z)


def norm_grads(x, w, b, z, dy, eps, kind):
    """dx, dweight, dbias, dgate of sum(y * dy)."""
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    xh, one = c * r, 1.0 if w is None else w
    dn, dz = dy, None
    if z is not None:
        s = sigmoid(z)
        dz = dy * (xh * one + (0.0 if b is None else b)) * (s + z * s * (1.0 - s))
        dn = dy * z * s
    d = dn * one
    dx = d - xh * (d * xh).mean(-1, keepdims=True)
    if kind == "layer":
        dx = dx - d.mean(-1, keepdims=True)
    return dx * r, (dn * xh).sum(0), dn.sum(0), dz


def cache_round(S, fmt):
    """What a stored state reads back as: every row over the smallest power of
    two (2^-126 at least) that keeps it within the format, on the format's grid."""
    top = 448.0 if fmt == "e4m3" else 127.0
    big = np.abs(S).max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        m, e = np.frexp(big / top)  # big / top = m 2^e, m in [0.5, 1); exactly 2^(e-1) at m = 0.5
        e = np.maximum(np.where(big == 0, -126, np.where(m == 0.5, e - 1, e)), -126)
        v = S * np.exp2(-e.astype(np.float64))
        grid = 1.0 if fmt == "int8" else np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
        out = np.rint(v / grid) * grid * np.exp2(e.astype(np.float64))
        # 2^128 is no fp32 number: the grid's next value towards zero instead
        out = np.where(np.abs(out) >= 2.0 ** 128, np.sign(out) * ((240.0 if fmt == "e4m3" else 63.0) * np.exp2(e.astype(np.float64))), out)
    return np.where(np.isfinite(big), out, np.nan)
