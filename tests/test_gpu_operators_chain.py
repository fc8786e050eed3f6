"""The operators together, as a layer uses them: the delta rule's prefill, its
heads normed and gated, a gated linear recurrence over the width, a norm; the
states put into the 8-bit cache, taken back, and one more token decoded. Every
tensor against the 64-bit plain forms (the delta rule's from the oracle).

Tolerances: the delta rule is held to 1e-4 of its largest value in fp32. A norm
of rows of size about 1 passes a relative error on by a factor of at most 4
(1 / rms, and the subtraction of the projection), and the recurrence with decays
up to 0.9 sums at most 10 tokens' errors, under gates below 1."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
import oracle
from gated_delta_rule_83_amd import inputs as gi
from tests import operators_ref as R
from tests.parity import rand_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, T, H, DK, DV = 2, 150, 2, 16, 32
W = H * DV


def weights(rng):
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    return dict(w1=1 + 0.1 * f(DV), z=f(B, T + 1, H, DV), a=rng.uniform(0.3, 0.9, (B, T + 1, W)).astype(np.float32),
                b=rng.uniform(0.1, 0.9, (B, T + 1, W)).astype(np.float32), w2=1 + 0.1 * f(W), b2=0.1 * f(W),
                h0=f(B, W))


def close(name, got, ref, tol):
    err = np.abs(R.f64(got) - ref).max() / np.abs(ref).max()
    print(f"[chain {name}] {err:.2e} (at most {tol:.0e})", flush=True)
    assert err <= tol, name


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_serving(fmt):
    rng = np.random.default_rng(1)
    d = rand_inputs(rng, B, T + 1, H, H, DK, DV)
    td = gi.to_torch(d, "f32", DEV)
    cut = lambda v, lo, hi: v[:, lo:hi].contiguous()
    u = {k: torch.tensor(v, device=DEV) for k, v in weights(rng).items()}
    f = {k: R.f64(v) for k, v in u.items()}
    args = [td[k] for k in ("q", "k", "v", "a", "b", "w")]

    o, S = g.chunk_forward(*(cut(v, 0, T) for v in args), td["S0"])
    n1 = g.norm_forward(o, u["w1"], None, cut(u["z"], 0, T), kind="rms")
    y, h = g.linear_forward(n1.view(B, T, W), cut(u["a"], 0, T), cut(u["b"], 0, T), u["h0"])
    out = g.norm_forward(y, u["w2"], u["b2"])

    ro, rS = oracle.forward(*(cut(v, 0, T) for v in args), td["S0"])
    r1 = R.norm(ro, f["w1"], None, f["z"][:, :T], 1e-5, "rms").reshape(B, T, W)
    ry, rh = zip(*(R.linear(r1[n], f["a"][n, :T], f["b"][n, :T], f["h0"][n], "channel") for n in range(B)))
    ry, rh = np.stack(ry), np.stack(rh)
    close("delta rule", o, ro, 1e-4)
    close("heads", n1.view(B, T, W), r1, 4e-4)
    close("recurrence", y, ry, 4e-3)
    close("out", out, R.norm(ry, f["w2"], f["b2"], None, 1e-5, "layer"), 1.6e-2)

    # both layers' states into their caches, back, and one more token
    slots = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    c1, s1 = g.state_cache_empty(5, H, DK, DV, device=DEV)
    c2, s2 = g.state_cache_empty(5, W // 16, 16, device=DEV)
    g.state_cache_store(S, slots, c1, s1, fmt=fmt)
    g.state_cache_store(h.view(B, W // 16, 16), slots, c2, s2, fmt=fmt)
    S2 = g.state_cache_load(c1, s1, slots, fmt=fmt)
    h2 = g.state_cache_load(c2, s2, slots, fmt=fmt).view(B, W)
    assert np.array_equal(R.f64(S2), R.cache_round(R.f64(S), fmt))
    assert np.array_equal(R.f64(h2), R.cache_round(R.f64(h).reshape(B, W // 16, 16), fmt).reshape(B, W))
    from_S, from_h = R.f64(S2), R.f64(h2)
    o1 = g.decode_step(*(cut(v, T, T + 1) for v in args), S2)
    n1 = g.norm_forward(o1, u["w1"], None, cut(u["z"], T, T + 1), kind="rms")
    y1 = g.linear_step(n1.view(B, W), u["a"][:, T].contiguous(), u["b"][:, T].contiguous(), h2)
    ro, rS = oracle.forward(*(cut(v, T, T + 1) for v in args), from_S.astype(np.float32))
    r1 = R.norm(ro, f["w1"], None, f["z"][:, T:], 1e-5, "rms").reshape(B, W)
    ry = f["a"][:, T] * from_h + f["b"][:, T] * r1
    close("decoded", o1, ro, 1e-4)
    close("stepped", y1, ry, 4e-3)
    assert torch.equal(h2, y1)


def test_training():
    """The loss's derivative along one direction of every input at once, against
    differences of the 64-bit chain (step 1e-4: its own error is 1e-8 of third
    derivatives). 1e-4 of the delta rule's gradients, times the factors above."""
    rng = np.random.default_rng(2)
    d = rand_inputs(rng, B, T, H, H, DK, DV)
    td = gi.to_torch(d, "f32", DEV)
    u = {k: torch.tensor(v[:, :T] if v.ndim >= 3 else v, device=DEV).contiguous() for k, v in weights(rng).items()}
    leaf = {k: v.clone().requires_grad_() for k, v in {**{"d" + k: td[k] for k in ("q", "k", "v", "a", "b", "w")}, **u}.items()}
    o, _ = g.gated_delta_rule(*(leaf["d" + k] for k in ("q", "k", "v", "a", "b", "w")), td["S0"])
    n1 = g.norm(o, leaf["w1"], None, leaf["z"], kind="rms")
    y, hT = g.gated_linear_recurrence(n1.view(B, T, W), leaf["a"], leaf["b"], leaf["h0"])
    out = g.norm(y, leaf["w2"], leaf["b2"])
    c1, c2 = rng.standard_normal((B, T, W)), rng.standard_normal((B, W))
    loss = (out.double() * torch.tensor(c1, device=DEV)).sum() + (hT.double() * torch.tensor(c2, device=DEV)).sum()
    grads = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))

    S0 = R.f64(td["S0"])
    f = {k: R.f64(v) for k, v in leaf.items()}

    def chain(q):
        ro, _ = oracle.forward(*(q["d" + k] for k in ("q", "k", "v", "a", "b", "w")), S0)
        r1 = R.norm(ro, q["w1"], None, q["z"], 1e-5, "rms").reshape(B, T, W)
        ry, rh = zip(*(R.linear(r1[n], q["a"][n], q["b"][n], q["h0"][n], "channel") for n in range(B)))
        return (R.norm(np.stack(ry), q["w2"], q["b2"], None, 1e-5, "layer") * c1).sum() + (np.stack(rh) * c2).sum()

    for k in leaf:
        v = rng.standard_normal(f[k].shape)
        num = (chain(dict(f, **{k: f[k] + 1e-4 * v})) - chain(dict(f, **{k: f[k] - 1e-4 * v}))) / 2e-4
        got = (R.f64(grads[k]) * v).sum()
        size = np.sqrt(((R.f64(grads[k]) * v) ** 2).sum())
        print(f"[chain gradient {k}] {got:.8g} {num:.8g}", flush=True)
        assert abs(got - num) <= 1.6e-2 * size + 1e-3


def test_second_derivatives_are_refused():
    x = torch.randn(2, 5, 8, device=DEV, requires_grad=True)
    a = torch.rand(2, 5, 8, device=DEV)
    for y in (g.gated_linear_recurrence(x, a, a)[0], g.norm(x)):
        with pytest.raises(RuntimeError, match="second derivatives"):
            torch.autograd.grad(y.sum(), x, create_graph=True)


def test_parts_of_a_graph_that_are_not_used():
    """Only the last state in the loss, frozen gates and weights, a gradient that is a view of one number."""
    x = torch.randn(2, 70, 8, device=DEV, requires_grad=True)
    a, b = torch.rand(2, 70, 8, device=DEV), torch.rand(2, 70, 8, device=DEV)
    h_T = g.gated_linear_recurrence(x, a, b)[1]
    dx = torch.autograd.grad(h_T.sum(), x)[0]
    ref = g.linear_backward(x.detach(), a, b, None, torch.zeros_like(a), torch.ones(2, 8, device=DEV))["dx"]
    assert torch.equal(dx, ref)
    w = torch.ones(8, device=DEV)
    z = torch.randn(2, 70, 8, device=DEV)
    dx = torch.autograd.grad(g.norm(x, w, w, z).sum(), x)[0]
    assert torch.equal(dx, g.norm_backward(x.detach(), w, w, z, torch.ones_like(z))["dx"])


def test_a_captured_training_step():
    """Forward and backward through autograd in one graph, replayed on new inputs, eager work between."""
    mk = lambda *s: torch.randn(*s, device=DEV)
    x, a, h0, w, dy = mk(1, 400, 64), torch.rand(1, 400, 64, device=DEV), mk(1, 64), mk(64), mk(1, 400, 64)

    def step():
        leaf = [t.detach().requires_grad_() for t in (x, a, h0, w)]
        o, h_T = g.gated_linear_recurrence(leaf[0], leaf[1], None, leaf[2], gates="tied")
        y = g.norm(o, leaf[3], kind="rms")
        return [y.detach(), h_T.detach(), *torch.autograd.grad((y, h_T), leaf, (dy, h0))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(mk(1, 400, 64))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for u, v in zip(got, step()):
            assert torch.equal(u, v), i


def test_calls_at_once_on_two_streams():
    """Chained recurrences of different sizes side by side: every call gives the bits it gives alone."""
    mk = lambda B, T, D: [torch.randn(B, T, D, device=DEV), torch.rand(B, T, D, device=DEV), torch.rand(B, T, D, device=DEV)]
    p, q = mk(1, 20000, 256), mk(3, 3000, 640)
    dO = torch.randn_like(q[0])
    alone = [g.linear_forward(*p)[0], *g.linear_backward(*q, None, dO).values()]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(5):
        got = []
        for _ in range(3):
            with torch.cuda.stream(s1):
                got.append((g.linear_forward(*p)[0], alone[0]))
            with torch.cuda.stream(s2):
                got += list(zip(g.linear_backward(*q, None, dO).values(), alone[1:]))
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in got), i
