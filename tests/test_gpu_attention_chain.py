"""The attention layer's operators together, as a model uses them: queries and
keys of a fused projection normed and rotated, a packed batch of prompts through
attention, their keys and values into pages, then token by token: normed,
rotated, stored, decoded. In fp32, every tensor against the 64-bit chain.

Tolerances (of the largest value): a rotated row is exact to 20 roundings, 1e-6;
scores of size s pass that on by a factor of at most 2 s (s below 10 here), so
the attention is held to 1e-4."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, HK, D, PAGE = 4, 2, 64, 16
EPS = float(np.float32(1e-6))


def freqs():
    return torch.tensor(1e4 ** (-np.arange(0, D, 2) / D), dtype=torch.float32, device=DEV)


def close(name, got, ref, tol):
    err = np.abs(R.f64(got) - ref).max() / np.abs(ref).max()
    print(f"[attention chain {name}] {err:.2e} (at most {tol:.0e})", flush=True)
    assert err <= tol, name


def split(x):
    return [t.unflatten(-1, (-1, D)) for t in x.split([H * D, HK * D, HK * D], -1)]


@pytest.mark.parametrize("window", [0, 20])
def test_serving(window):
    rng = np.random.default_rng(1)
    lens, steps = [70, 1, 33], 3
    N, T = len(lens), sum(lens)
    mk = lambda *s: torch.tensor(rng.standard_normal(s).astype(np.float32), device=DEV)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    wq, wk, f = 1 + 0.1 * mk(D), 1 + 0.1 * mk(D), freqs()
    prompt, later = mk(T, (H + 2 * HK) * D), [mk(N, 1, (H + 2 * HK) * D) for _ in range(steps)]
    cu = np.concatenate(([0], np.cumsum(lens)))
    pos = np.concatenate([np.arange(n) for n in lens])
    need = [-(-(n + steps) // PAGE) for n in lens]
    order = rng.permutation(sum(need) + 2)
    table, at = np.full((N, max(need)), -1), 0
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
    kc, vc = g.kv_cache_empty(sum(need) + 2, HK, D, page=PAGE, dtype=torch.float32, device=DEV)
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    pages = ints(table)

    q, k, v = split(prompt)
    q, k = g.rotary_forward(q, k, ints(pos), f, wq, wk, eps=EPS)
    o, _ = g.attention_forward_varlen(q, k, v, ints(cu), window=window)
    g.kv_cache_store(k, v, pages, ints(lens), kc, vc, cu_seqlens=ints(cu))
    decoded = []
    for i, x in enumerate(later):
        q1, k1, v1 = split(x)
        q1, k1 = g.rotary_forward(q1, k1, ints([[n + i] for n in lens]), f, wq, wk, eps=EPS)
        ln = ints([n + i + 1 for n in lens])
        g.kv_cache_store(k1, v1, pages, ln, kc, vc)
        decoded.append(g.attention_decode(q1, kc, vc, pages, ln, window=window))
    torch.cuda.synchronize()

    F, scale = f.cpu().numpy(), float(np.float32(D ** -0.5))
    for n in range(N):
        rows = np.concatenate([R.f64(prompt[cu[n]:cu[n + 1]])] + [R.f64(x[n]) for x in later])
        p = np.arange(len(rows))
        rq = R.rotary(rows[:, :H * D].reshape(-1, H, D), R.f64(wq), p, F, EPS, True, "halves")
        rk = R.rotary(rows[:, H * D:(H + HK) * D].reshape(-1, HK, D), R.f64(wk), p, F, EPS, True, "halves")
        rv = rows[:, (H + HK) * D:].reshape(-1, HK, D)
        ro = np.stack([R.attention(rq[:, h], rk[:, h // 2], rv[:, h // 2], None, scale, True, window, torch.float32)["o"][0]
                       for h in range(H)], 1)
        close(f"q {n}", q[cu[n]:cu[n + 1]], rq[:lens[n]], 2e-6)
        close(f"k {n}", k[cu[n]:cu[n + 1]], rk[:lens[n]], 2e-6)
        close(f"prompt {n}", o[cu[n]:cu[n + 1]], ro[:lens[n]], 1e-4)
        for i in range(steps):
            close(f"token {i} of {n}", decoded[i][n, 0], ro[lens[n] + i], 1e-4)


def layer(x, wq, wk, pos, f, window=0):
    q, k, v = split(x)
    q, k = g.rotary(q, k, pos, f, wq, wk, eps=1e-3)
    return g.attention(q, k, v, window=window)


@pytest.mark.parametrize("window", [0, 30])
def test_training(window):
    """The loss's derivative along a direction of every input, against differences of the 64-bit chain."""
    rng = np.random.default_rng(2)
    B, T = 2, 90
    mk = lambda *s: torch.tensor(rng.standard_normal(s).astype(np.float32), device=DEV)  # noqa: E731
    x, wq, wk, f, dO = mk(B, T, (H + 2 * HK) * D), 1 + 0.1 * mk(D), 1 + 0.1 * mk(D), freqs(), mk(B, T, H, D)
    pos = torch.arange(T, dtype=torch.int32, device=DEV).expand(B, T).contiguous()
    leaf = [t.clone().requires_grad_() for t in (x, wq, wk)]
    grads = torch.autograd.grad(layer(*leaf, pos, f, window), leaf, dO)
    F, P, G, eps, scale = f.cpu().numpy(), np.arange(T), R.f64(dO), float(np.float32(1e-3)), float(np.float32(D ** -0.5))

    def loss(v):
        total = 0.0
        for b in range(B):
            rq = R.rotary(v[0][b][:, :H * D].reshape(T, H, D), v[1], P, F, eps, True, "halves")
            rk = R.rotary(v[0][b][:, H * D:(H + HK) * D].reshape(T, HK, D), v[2], P, F, eps, True, "halves")
            rv = v[0][b][:, (H + HK) * D:].reshape(T, HK, D)
            total += sum((R.attention(rq[:, h], rk[:, h // 2], rv[:, h // 2], None, scale, True, window, torch.float32)["o"][0]
                          * G[b, :, h]).sum() for h in range(H))
        return total

    base = [R.f64(t) for t in (x, wq, wk)]
    for i, nm in enumerate(("x", "wq", "wk")):
        w = rng.standard_normal(base[i].shape)
        step = lambda e: loss([t + e * w if j == i else t for j, t in enumerate(base)])  # noqa: E731, B023
        num, got = (step(1e-5) - step(-1e-5)) / 2e-5, (R.f64(grads[i]) * w).sum()
        size = np.sqrt(((R.f64(grads[i]) * w) ** 2).sum())
        print(f"[attention chain gradient {nm}] {got:.8g} {num:.8g}", flush=True)
        # each gradient value to 1e-4 of its size, their errors independent; the differences' own error
        assert abs(got - num) <= 1e-4 * size + 1e-6 * (1 + abs(num))


def test_a_captured_training_step():
    """Forward and backward through autograd in one graph, replayed on new inputs, eager work between."""
    mk = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    x, wq, wk, f, dO = mk(1, 200, (H + 2 * HK) * D), mk(D), mk(D), freqs(), mk(1, 200, H, D)
    pos = torch.arange(200, dtype=torch.int32, device=DEV)[None]

    def step():
        leaf = [t.detach().requires_grad_() for t in (x, wq, wk)]
        o = layer(*leaf, pos, f)
        return [o.detach(), *torch.autograd.grad(o, leaf, dO)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(mk(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for u, v in zip(got, step()):
            assert torch.equal(u, v), i


def test_calls_at_once_on_two_streams():
    """Different problems side by side: every call gives the bits it gives alone."""
    mk = lambda *s: torch.randn(*s, device=DEV).to(torch.bfloat16)  # noqa: E731
    a, b = [mk(1, 2000, h, 128) for h in (8, 2, 2)], [mk(3, 300, h, 64) for h in (4, 4, 4)]
    da, db = torch.randn_like(a[0]), torch.randn_like(b[0])

    def both(t, d):
        o, lse = g.attention_forward(*t)
        return [o, lse, *g.attention_backward(*t, o, lse, d).values()]

    alone = both(a, da), both(b, db)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(5):
        got = []
        for _ in range(3):
            with torch.cuda.stream(s1):
                got += list(zip(both(a, da), alone[0]))
            with torch.cuda.stream(s2):
                got += list(zip(both(b, db), alone[1]))
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in got), i


def test_second_derivatives_are_refused():
    x = torch.randn(1, 8, 2, 64, device=DEV, requires_grad=True)
    pos = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    for y in (g.attention(x, x, x), g.rotary(x, None, pos, freqs())[0]):
        with pytest.raises(RuntimeError, match="second derivatives"):
            torch.autograd.grad(y.sum(), x, create_graph=True)


def test_parts_of_a_graph_that_are_not_used():
    """Frozen weights, a gradient that is a view of one number, only the keys in the loss, the same tensor thrice."""
    x, pos, f = torch.randn(2, 40, 2, 64, device=DEV), torch.arange(80, dtype=torch.int32, device=DEV).view(2, 40), freqs()
    w = torch.ones(64, device=DEV)
    leaf = x.clone().requires_grad_()
    _, k = g.rotary(x, leaf, pos, f, w, w)
    dk, = torch.autograd.grad(k.sum(), leaf)
    want = g.rotary_backward(x, x, pos, f, w, w, torch.zeros_like(x), torch.ones_like(x))["dk"]
    assert torch.equal(dk, want)
    dx, = torch.autograd.grad(g.attention(leaf, leaf, leaf).sum(), leaf)
    o, lse = g.attention_forward(x, x, x)
    gr = g.attention_backward(x, x, x, o, lse, torch.ones_like(x))
    torch.cuda.synchronize()
    assert torch.allclose(dx, gr["dq"] + gr["dk"] + gr["dv"], rtol=0, atol=4 * R.U * float(sum(t.abs().max() for t in gr.values())))
