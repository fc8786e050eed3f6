"""Head norm and rotation by position (gdn2_rotary_*) against the 64-bit plain form.

Bounds. The mean square is off by (d / 16 + 12) u of itself (a row lies on up to
64 lanes), its root and reciprocal by 3 more roundings; a normed and weighted
value by 3 more; a turned one is the sum of two products with a sine and cosine
off by 4 u (the angle within a turn is rounded to 2^-25 of a turn). The backward's
mean of products likewise; weights' sums over n rows by (n / 64 + 64) u of their
terms' magnitudes."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = R.U


def freqs(rot, base=1e6):
    return torch.tensor(base ** (-np.arange(0, rot, 2) / max(rot, 1)), dtype=torch.float32, device=DEV)


def rand(rng, *shape, dtype="bf16"):
    return torch.tensor(rng.standard_normal(shape).astype(np.float32)).to(R.TYPES[dtype]).to(DEV)


def one(name, x, w, pos, f, eps, norm, pairs, y, dy=None, dx=None, dw=None):
    h = R.half(x.dtype)
    X, W, F, p = R.f64(x), None if w is None else R.f64(w), f.cpu().numpy(), pos.cpu().numpy()
    d = X.shape[-1]
    ones = np.ones(d) if W is None else W
    r = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + eps) if norm else np.ones_like(X[..., :1])
    K = ((d / 16 + 12) / 2 + 3 if norm else 0) * U
    rot = 2 * len(F)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if pairs == "halves" else (slice(0, rot, 2), slice(1, rot, 2))

    def pair(v):  # |v_a| + |v_b| in both places of a pair
        t = np.abs(v).copy()
        t[..., a], t[..., b] = (np.abs(v[..., a]) + np.abs(v[..., b]),) * 2
        return t

    def hold(nm, got, ref, tol):
        hh = R.half(got.dtype)
        R.hold(f"{name} {nm}", got, ref, tol + (hh + 2 * U) * (np.abs(ref) + tol) + 1e-30)

    ref = R.rotary(X, W, p, F, eps, norm, pairs, None if dy is None else R.f64(dy))
    u = X * r * ones
    hold("y", y, ref if dy is None else ref[0], (K + 3 * U + 10 * U) * pair(u))
    if dy is None:
        return
    G = R.f64(dy)
    tdu = 10 * U * pair(G)
    du = R.rotary(G, None, -p, F, 0.0, False, pairs)
    D, tD, xh = du * ones, (tdu + 2 * U * np.abs(du)) * np.abs(ones), X * r
    if norm:
        mean = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
        m = mean(np.abs(D * xh))
        tm = mean(tD * np.abs(xh)) + (K + 2 * U) * m + (d / 16 + 14) * U * m
        tol = r * (tD + np.abs(xh) * (tm + (K + 4 * U) * m)) + (K + 6 * U) * r * (np.abs(D) + np.abs(xh) * m)
    else:
        tol = tD
    hold("dx", dx, ref[1], tol + h * 0)
    if dw is not None:
        n = X.shape[0] * X.shape[1]
        hold("dw", dw, ref[2], (((n / 64 + 64) * U + K + 2 * U) * np.abs(du * xh) + tdu * np.abs(xh)).sum((0, 1)))


SHAPES = [(1, 1, 1, 2, 2), (3, 2, 1, 8, 8), (5, 4, 2, 16, 8), (7, 3, 3, 32, 32), (130, 4, 1, 64, 64), (33, 16, 2, 128, 128),
          (9, 5, 1, 128, 64), (6, 2, 2, 96, 48), (4, 3, 1, 80, 40), (5, 2, 1, 256, 256), (3, 2, 1, 256, 64), (5, 2, 1, 10, 4),
          (4, 2, 1, 62, 62), (3, 1, 1, 320, 320), (2, 1, 1, 1024, 512), (3, 2, 0, 64, 0), (2500, 2, 1, 64, 32)]


@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("norm,weights", [(True, True), (True, False), (False, False), (False, True)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("N,H,Hk,d,rot", SHAPES)
def test_forward_and_gradients(N, H, Hk, d, rot, pairs, norm, weights, dtype, wtype):
    rng = np.random.default_rng(N + d + rot)
    q, dq_out = rand(rng, N, H, d, dtype=dtype), rand(rng, N, H, d, dtype=dtype)
    k, dk_out = (rand(rng, N, Hk, d, dtype=dtype), rand(rng, N, Hk, d, dtype=dtype)) if Hk else (None, None)
    qw = (1 + 0.2 * rand(rng, d, dtype="f32")).to(R.TYPES[wtype]) if weights else None
    kw = rand(rng, d, dtype=wtype) if weights and Hk else None
    pos = torch.tensor(rng.integers(0, 5000, N), dtype=torch.int32, device=DEV)
    f, eps = freqs(rot), float(np.float32(1e-5))
    qo, ko = g.rotary_forward(q, k, pos, f, qw, kw, eps=eps, norm=norm, pairs=pairs)
    gr = g.rotary_backward(q, k, pos, f, qw, kw, dq_out, dk_out, eps=eps, norm=norm, pairs=pairs)
    torch.cuda.synchronize()
    one("rotary q", q, qw, pos, f, eps, norm, pairs, qo, dq_out, gr["dq"], gr["dq_weight"])
    if Hk:
        one("rotary k", k, kw, pos, f, eps, norm, pairs, ko, dk_out, gr["dk"], gr["dk_weight"])
    else:
        assert ko is None and gr["dk"] is None


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_far_positions(pairs):
    """Positions to the ends of int32, negative ones too: as exact as near ones."""
    rng = np.random.default_rng(1)
    at = [0, 1, -1, 1 << 20, (1 << 24) + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31]
    q = rand(rng, len(at), 2, 64, dtype="f32")
    pos = torch.tensor(at, dtype=torch.int32, device=DEV)
    y, _ = g.rotary_forward(q, None, pos, freqs(64), norm=False, pairs=pairs)
    torch.cuda.synchronize()
    one("rotary far", q, None, pos, freqs(64), 0.0, False, pairs, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_of_a_fused_projection_and_unaligned_tensors(dtype):
    B, T, H, Hk, d = 2, 21, 4, 2, 64
    rng = np.random.default_rng(2)
    qkv = rand(rng, B, T, (H + 2 * Hk) * d, dtype=dtype)
    q, k, _ = (x.unflatten(-1, (-1, d)) for x in qkv.split([H * d, Hk * d, Hk * d], -1))
    w, f = rand(rng, d, dtype="f32"), freqs(d)
    pos = torch.arange(T, dtype=torch.int32, device=DEV).expand(B, T).contiguous()
    qo, ko = g.rotary_forward(q, k, pos, f, w, w)
    q2, k2 = g.rotary_forward(q.contiguous(), k.contiguous(), pos, f, w, w)
    # one element off: single values
    off = torch.empty(q.numel() + 1, dtype=q.dtype, device=DEV)
    qu = off[1:].view(q.shape)
    qu.copy_(q)
    q3, k3 = g.rotary_forward(qu, k, pos, f, w, w)
    torch.cuda.synchronize()
    assert qo.is_contiguous() and torch.equal(qo, q2) and torch.equal(ko, k2)
    # its sums run in another order: within the bound, not to the bit
    for nm, x, y in (("q", qu, q3), ("k", k, k3)):
        one(f"rotary unaligned {nm}", x.flatten(0, 1), w, pos.flatten(), f, float(np.float32(1e-6)), True, "halves", y.flatten(0, 1))
    leaf = qkv.detach().requires_grad_()
    ql, kl, _ = (x.unflatten(-1, (-1, d)) for x in leaf.split([H * d, Hk * d, Hk * d], -1))
    wl = w.clone().requires_grad_()
    a, b = g.rotary(ql, kl, pos, f, wl, wl)
    grad, gw = torch.autograd.grad((a, b), (leaf, wl), (torch.ones_like(a), torch.ones_like(b)))
    gr = g.rotary_backward(q.contiguous(), k.contiguous(), pos, f, w, w, torch.ones_like(a), torch.ones_like(b))
    torch.cuda.synchronize()
    assert torch.equal(grad[..., :H * d], gr["dq"].flatten(-2)) and torch.equal(grad[..., H * d:(H + Hk) * d], gr["dk"].flatten(-2))
    assert (grad[..., (H + Hk) * d:] == 0).all() and torch.equal(gw, gr["dq_weight"] + gr["dk_weight"])


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    N, H, Hk, d, rot = 6, 2, 1, 32, 16
    q, k, w = rand(rng, N, H, d, dtype="f32"), rand(rng, N, Hk, d, dtype="f32"), 1 + 0.3 * rand(rng, d, dtype="f32")
    pos, f, eps = torch.arange(N, dtype=torch.int32, device=DEV), freqs(rot), float(np.float32(1e-3))
    gq, gk = rand(rng, N, H, d, dtype="f32"), rand(rng, N, Hk, d, dtype="f32")
    leaf = [x.clone().requires_grad_() for x in (q, k, w)]
    out = g.rotary(leaf[0], leaf[1], pos, f, leaf[2], leaf[2], eps=eps)
    grads = torch.autograd.grad(out, leaf, (gq, gk))
    base = [R.f64(x) for x in (q, k, w)]
    P, F = pos.cpu().numpy(), f.cpu().numpy()
    loss = lambda v: ((R.rotary(v[0], v[2], P, F, eps, True, "halves") * R.f64(gq)).sum()  # noqa: E731
                      + (R.rotary(v[1], v[2], P, F, eps, True, "halves") * R.f64(gk)).sum())
    for i in range(3):
        t = rng.standard_normal(base[i].shape)
        step = lambda e: loss([x + e * t if j == i else x for j, x in enumerate(base)])  # noqa: E731, B023
        num, got = (step(1e-5) - step(-1e-5)) / 2e-5, (R.f64(grads[i]) * t).sum()
        assert abs(got - num) <= 64 * U * np.abs(R.f64(grads[i])).max() * np.abs(t).sum() + 1e-6 * (1 + abs(num))


def test_no_tokens_and_parts_not_wanted():
    e = torch.empty(0, 4, 64, device=DEV)
    w, f, pos = torch.ones(64, device=DEV), freqs(64), torch.empty(0, dtype=torch.int32, device=DEV)
    q, k = g.rotary_forward(e, e[:, :2].contiguous(), pos, f, w, w)
    gr = g.rotary_backward(e, e, pos, f, w, w, e, e)
    torch.cuda.synchronize()
    assert q.shape == (0, 4, 64) and (gr["dq_weight"] == 0).all() and (gr["dk_weight"] == 0).all()
    rng = np.random.default_rng(4)
    q = rand(rng, 10, 4, 64)
    pos = torch.arange(10, dtype=torch.int32, device=DEV)
    full = g.rotary_backward(q, q, pos, f, w, w, q, q)
    part = g.rotary_backward(q, q, pos, f, w, w, q, q, want_weights=False)
    torch.cuda.synchronize()
    assert part["dq_weight"] is None and torch.equal(full["dq"], part["dq"]) and torch.equal(full["dk"], part["dk"])


def test_a_bad_row_stays_alone_and_graphs_repeat():
    rng = np.random.default_rng(5)
    q, k, w, f = rand(rng, 300, 4, 128), rand(rng, 300, 2, 128), rand(rng, 128, dtype="f32"), freqs(128)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)
    a, b = g.rotary_forward(q, k, pos, f, w, w)
    gr = g.rotary_backward(q, k, pos, f, w, w, a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a2, b2 = g.rotary_forward(q, k, pos, f, w, w)
        gr2 = g.rotary_backward(q, k, pos, f, w, w, a, b)
    for i in range(3):
        for t in (a2, b2, *gr2.values()):
            t.fill_(float("nan"))
        graph.replay()
        g.rotary_forward(q, k, pos, f, w, w)
        torch.cuda.synchronize()
        assert torch.equal(a, a2) and torch.equal(b, b2) and all(torch.equal(gr[n], gr2[n]) for n in gr), i
    q[7, 2, 9] = float("inf")
    a3, b3 = g.rotary_forward(q, k, pos, f, w, w)
    torch.cuda.synchronize()
    keep = torch.ones(300, 4, dtype=torch.bool, device=DEV)
    keep[7, 2] = False
    assert torch.equal(a[keep], a3[keep]) and torch.equal(b, b3) and torch.isnan(a3[7, 2]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,Hk,d", [(5, 4, 1, 64), (40, 16, 2, 128), (3000, 3, 2, 64), (7, 1, 1, 32), (9, 2, 1, 256), (4, 2, 1, 62)])
def test_no_epsilon(N, H, Hk, d, dtype):
    """eps = 0, and heads that leave lanes of a wave without one: a weight's gradient takes nothing from those."""
    rng = np.random.default_rng(N + d)
    q, k, gq, gk = (rand(rng, N, h, d, dtype=dtype) for h in (H, Hk, H, Hk))
    qw, kw, f = 1 + 0.2 * rand(rng, d, dtype="f32"), rand(rng, d, dtype="f32"), freqs(d)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    qo, ko = g.rotary_forward(q, k, pos, f, qw, kw, eps=0.0)
    gr = g.rotary_backward(q, k, pos, f, qw, kw, gq, gk, eps=0.0)
    torch.cuda.synchronize()
    one("rotary eps 0 q", q, qw, pos, f, 0.0, True, "halves", qo, gq, gr["dq"], gr["dq_weight"])
    one("rotary eps 0 k", k, kw, pos, f, 0.0, True, "halves", ko, gk, gr["dk"], gr["dk_weight"])


PI = 31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679821  # times 10^103


def turns_of(position, frequency):
    """The fraction of a turn, -1/2 .. 1/2, of position * frequency, by whole numbers alone."""
    m = int(float(frequency) * 2 ** 40)  # exact: frequencies of 24 bits from 2^-16 on
    assert m == float(frequency) * 2 ** 40
    scaled = position * m * 2 ** 160 * 10 ** 103 // (2 * PI)  # turns * 2^200
    scaled = (scaled + 2 ** 199) % 2 ** 200 - 2 ** 199
    return scaled / 2 ** 200


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("d", [64, 62])
def test_far_angles_are_as_exact_as_near_ones(d, pairs):
    """Sines and cosines themselves (pairs of 1 and 0) at positions near 2^31. The fraction of a turn is rounded once,
    x half turns by u |x|, and a sine or cosine is off by two units in the last place, 4 u of itself: where the angle is
    near a whole turn this sees errors far below u."""
    rng = np.random.default_rng(6)
    N, half = 96, d // 2
    pos = np.concatenate((rng.integers(2 ** 31 - 2 ** 20, 2 ** 31, N // 2), rng.integers(-2 ** 31, -2 ** 31 + 2 ** 20, N // 4),
                          rng.integers(0, 100, N // 4)))
    f = rng.uniform(0.5, 1, half).astype(np.float32)
    f[half // 2:] *= np.float32(2.0) ** -rng.integers(0, 15, half - half // 2)
    q = torch.zeros(N, 1, d, device=DEV)
    a, b = (slice(0, half), slice(half, d)) if pairs == "halves" else (slice(0, d, 2), slice(1, d, 2))
    q[..., a] = 1
    y, _ = g.rotary_forward(q, None, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(f, device=DEV), norm=False,
                            pairs=pairs)
    torch.cuda.synchronize()
    x = 2 * np.array([[turns_of(int(p), v) for v in f] for p in pos])
    c, s = np.cos(np.pi * x), np.sin(np.pi * x)
    assert np.abs(x[:N // 2]).min() < 2.0 ** -8  # some near a whole turn
    Y = R.f64(y)[:, 0]
    R.hold("far sines", torch.tensor(Y[:, b]), s, U * (np.pi * np.abs(x) + 4 * np.abs(s)) + 1e-15)
    R.hold("far cosines", torch.tensor(Y[:, a]), c, U * (np.pi * np.abs(x * s) + 4 * np.abs(c)) + 1e-15)
