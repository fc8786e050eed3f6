"""Plain 64-bit forms of the attention layer's operators and error bounds for
them (test infrastructure).

Bounds. u = 2^-24 is one rounding to fp32, half(t) one to the type t. A product
of d terms summed in fp32 in any order is off by at most (d + 8) u of the sum of
its terms' magnitudes (8 for what a wave or the matrix cores join). A score s is
off by ds = that times scale + 6 u |s| (scale * log2 e, its product and the
difference are a rounding each), so a probability is off by the factor
e^(2 ds) + 4 u at most: rel = 2.1 ds + 8 u while ds < 0.02. In bf16 each
probability, and each gradient of a score, is rounded once more as an operand."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def half(dtype) -> float:
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def visible(nq, nk, causal, window):
    at, j = np.arange(nq)[:, None] + nk - nq, np.arange(nk)[None]
    see = np.ones((nq, nk), bool)
    if causal:
        see &= j <= at
    if window:
        see &= j > at - window
    return see


def attention(q, k, v, dO, scale, causal, window, dtype):
    """One sequence, one query head: q, dO [nq, d], k, v [nk, d] in 64 bits (dO
    None: forward alone). A dict name -> (value, bound)."""
    nq, nk, d = q.shape[0], k.shape[0], q.shape[1]
    h = half(dtype)
    see = visible(nq, nk, causal, window)
    s = scale * (q @ k.T)
    ds_ = scale * (d + 8) * U * (np.abs(q) @ np.abs(k).T) + 6 * U * np.abs(s)
    sm = np.where(see, s, -np.inf)
    some = see.any(1)
    top = np.where(some, sm.max(1, initial=-np.inf), 0.0)
    e = np.exp(sm - top[:, None])
    total = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(some, top + np.log(np.where(some, total, 1.0)), -np.inf)
    p = e / np.where(some, total, 1.0)[:, None]
    rel = 2.1 * ds_ + 8 * U
    relp = rel + (p * rel).sum(1, keepdims=True) + (nk / 16 + 16) * U  # and the sum's
    o = p @ v
    to = (p * (relp + h)) @ np.abs(v) + (nk + 16) * U * (p @ np.abs(v))
    dl = np.where(some, (p * rel).sum(1) + (nk / 16 + 16) * U + 8 * U * np.abs(np.where(some, lse, 0)) + 4 * U, 0.0)
    last = lambda x, t: t + (h + 2 * U) * (np.abs(x) + t)  # noqa: E731
    out = {"o": (o, last(o, to)), "lse": (lse, dl)}
    if dO is None:
        return out
    # the probabilities again, from lse as the forward left it
    relb = rel + dl[:, None] + 8 * U
    dp = dO @ v.T
    tdp = (d + 8) * U * (np.abs(dO) @ np.abs(v).T)
    delta = (dO * o).sum(1)
    tdelta = (np.abs(dO) * last(o, to)).sum(1) + (d + 8) * U * (np.abs(dO) * (np.abs(o) + to)).sum(1)
    ds = p * (dp - delta[:, None])
    tds = np.abs(ds) * (relb + h + 4 * U) + p * (1 + h) * (tdp + tdelta[:, None] + 2 * U * (np.abs(dp) + np.abs(delta)[:, None]))
    dq = scale * ds @ k
    tq = scale * (tds @ np.abs(k) + (nk + 16) * U * (np.abs(ds) @ np.abs(k)))
    dk = scale * ds.T @ q
    tk = scale * (tds.T @ np.abs(q) + (nq + 16) * U * (np.abs(ds).T @ np.abs(q)))
    dv = p.T @ dO
    tv = (p * (relb + h)).T @ np.abs(dO) + (nq + 16) * U * (p.T @ np.abs(dO))
    out.update(dq=(dq, last(dq, tq)), dk=(dk, tk), dv=(dv, tv))  # dk, dv: still to be summed over heads
    return out


def grouped(q, k, v, dO, scale, causal, window, dtype):
    """One sequence: q, dO [nq, H, d], k, v [nk, H_kv, d] (tensors)."""
    Q, K, V = f64(q), f64(k), f64(v)
    G_ = None if dO is None else f64(dO)
    H, Hkv, h = Q.shape[1], K.shape[1], half(dtype)
    group = H // Hkv
    names = ("o", "lse") if dO is None else ("o", "lse", "dq", "dk", "dv")
    shape = {"o": Q.shape, "lse": (H, Q.shape[0]), "dq": Q.shape, "dk": K.shape, "dv": K.shape}
    out = {n: (np.zeros(shape[n]), np.zeros(shape[n])) for n in names}
    for head in range(H):
        kv = head // group
        r = attention(Q[:, head], K[:, kv], V[:, kv], None if G_ is None else G_[:, head], scale, causal, window, dtype)
        for n in names:
            at = head if n == "lse" else (slice(None), kv if n in ("dk", "dv") else head)
            for i in range(2):
                out[n][i][at] += r[n][i]
    for n in ("dk", "dv"):
        if n in out:  # the sum over the group's heads, and the output's rounding
            x, t = out[n]
            t = t + 2 * group * U * (np.abs(x) + t)
            out[n] = (x, t + (h + 2 * U) * (np.abs(x) + t))
    return out


def hold(name, got, ref, bound):
    """Every value within its bound; infinities and NaN exactly where they belong."""
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(g[~fine], ref[~fine], equal_nan=True), name
    err = np.abs(g[fine] - ref[fine])
    worst = float((err / np.maximum(bound[fine], 1e-300)).max()) if err.size else 0.0
    print(f"[{name}] worst error over its bound {worst:.3f}", flush=True)
    assert np.isfinite(g[fine]).all() and worst <= 1.0, (name, worst)


# ------------------------------------------------------------------ head norm and rotation
def rotary(x, w, pos, inv_freq, eps, norm, pairs, dy=None):
    """x [N, H, d] in 64 bits. y, or (y, dx, dw)."""
    rot = 2 * len(inv_freq)
    angle = pos[:, None].astype(np.float64) * inv_freq.astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if pairs == "halves" else (slice(0, rot, 2), slice(1, rot, 2))

    def turn(u, sign):
        y = u.copy()
        y[..., a], y[..., b] = u[..., a] * c - sign * u[..., b] * s, u[..., b] * c + sign * u[..., a] * s
        return y

    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else np.ones_like(x[..., :1])
    xh = x * r
    y = turn(xh * (1.0 if w is None else w), 1.0)
    if dy is None:
        return y
    du = turn(dy, -1.0)
    d = du * (1.0 if w is None else w)
    dx = r * (d - xh * (d * xh).mean(-1, keepdims=True)) if norm else d
    return y, dx, (du * xh).sum((0, 1))
