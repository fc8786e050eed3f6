"""The gated linear recurrence (gdn2_linear_*) against its 64-bit plain form.

Tolerances. With every decay at most AMAX, an error made at one token is
carried on by at most 1 / (1 - AMAX) tokens' worth. A token makes at most 16
roundings of half an fp32 step on terms no larger than the largest |h| (four of
the activation's exponential, sum and reciprocal, one of the product b x, one
of the step, and those of the scan's compositions, at most log2(128) + 3). So
|h - h_ref| <= E32 * max|h| with E32 = 16 * 2^-24 / (1 - AMAX), the same for the
adjoints, and a product of two such values is off by the sum of both. An output
in bf16 is off by one more rounding of itself."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
AMAX = 0.98
E32 = 16 * R.U32 / (1 - AMAX)


def problem(rng, lead, D, n, form, dtype, a_hi=AMAX):
    """Tensors of a problem: x, a, b, h0, dO, dh_T (tokens lead + (D,), n states)."""
    dt = R.TORCH[dtype]
    mk = lambda v, d: torch.tensor(np.asarray(v, np.float32)).to(d).to(DEV)
    A = rng.uniform(0.3, a_hi, lead + (D,))
    Bv = rng.standard_normal(lead + (D,))
    if form in ("preact", "tied_preact"):  # log(1 / a - 1), rounded towards smaller decays
        pre = np.log(1.0 / A - 1.0)
        a, b = mk(pre + 2.0 ** -7 * np.abs(pre), dt), mk(Bv, dt)
    else:
        a, b = mk(A, torch.float32), mk(R.sigmoid(Bv), torch.float32)
    if form in ("tied", "tied_preact"):
        b = None
    return dict(x=mk(rng.standard_normal(lead + (D,)), dt), a=a, b=b, h0=mk(rng.standard_normal((n, D)), torch.float32),
                dO=mk(rng.standard_normal(lead + (D,)), dt), dhT=mk(rng.standard_normal((n, D)), torch.float32))


def close(name, got, ref, scale, dtype=torch.float32, k=1.0):
    err = np.abs(R.f64(got) - ref)
    tol = k * E32 * scale + (0 if dtype == torch.float32 else R.half(dtype)) * (np.abs(ref) + k * E32 * scale)
    worst = float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0
    print(f"[linear {name}] worst error over its bound {worst:.3f}", flush=True)
    assert np.isfinite(R.f64(got)).all() and worst <= 1.0, name


def check(p, spans, form, o, h_T, gr=None, packed=False):
    """Every sequence of `spans` (index of its tokens, state row) against the plain form."""
    f = {k: R.f64(v) for k, v in p.items()}
    for at, n in spans:
        args = [f["x"][at], f["a"][at], None if f["b"] is None else f["b"][at], f["h0"][n]]
        ro, rT = R.linear(*args, form)
        hs = max(np.abs(ro).max() if ro.size else 0.0, np.abs(f["h0"][n]).max())
        close(f"o {n}", o[at], ro, hs, o.dtype)
        close(f"h_T {n}", h_T[n], rT, hs)
        if gr is None:
            continue
        dx, da, db, dh0, ad = R.linear_grads(*args, f["dO"][at], f["dhT"][n], form)
        gs = max(np.abs(ad).max() if ad.size else 0.0, np.abs(f["dhT"][n]).max())
        xs = np.abs(args[0]).max() if ro.size else 0.0
        gt = p["a"].dtype
        close(f"dx {n}", gr["dx"][at], dx, gs, o.dtype)
        close(f"da {n}", gr["da"][at], da, gs * (hs + xs), gt, 2.0)
        if db is not None:
            close(f"db {n}", gr["db"][at], db, gs * xs, gt, 2.0)
        close(f"dh0 {n}", gr["dh0"][n], dh0, gs)


SIZES = [(1, 1, 1), (2, 2, 3), (1, 127, 4), (3, 128, 64), (2, 129, 65), (1, 300, 130), (2, 1000, 68), (1, 2500, 260)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", R.FORMS)
@pytest.mark.parametrize("B,T,D", SIZES)
def test_sequences_and_gradients(B, T, D, form, dtype):
    p = problem(np.random.default_rng(T * 100 + D), (B, T), D, B, form, dtype)
    o, h_T, ck = g.linear_forward(p["x"], p["a"], p["b"], p["h0"], want_checkpoints=True, gates=form)
    gr = g.linear_backward(p["x"], p["a"], p["b"], p["h0"], p["dO"], p["dhT"], ck=ck, gates=form)
    torch.cuda.synchronize()
    check(p, [(n, n) for n in range(B)], form, o, h_T, gr)
    # the states computed again instead of saved: the same numbers
    again = g.linear_backward(p["x"], p["a"], p["b"], p["h0"], p["dO"], p["dhT"], gates=form)
    for k in gr:
        assert gr[k] is None if again[k] is None else torch.equal(gr[k], again[k]), k
    # no initial state, no last state's gradient
    z = dict(p, h0=torch.zeros_like(p["h0"]), dhT=torch.zeros_like(p["dhT"]))
    o, h_T = g.linear_forward(p["x"], p["a"], p["b"], gates=form)
    gr = g.linear_backward(p["x"], p["a"], p["b"], None, p["dO"], gates=form)
    check(z, [(n, n) for n in range(B)], form, o, h_T, gr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", R.FORMS)
@pytest.mark.parametrize("lens,D", [([5], 4), ([0, 3, 0, 0, 125, 130, 0], 64), ([1] * 300, 68), ([700, 1, 1, 513, 128], 33),
                                    ([0, 0], 8)])
def test_packed(lens, D, form, dtype):
    lead, tail = 2, 3  # rows before the first and behind the last sequence
    T = lead + sum(lens) + tail
    cu = np.concatenate([[lead], lead + np.cumsum(lens)]).astype(np.int32)
    N = len(lens)
    p = problem(np.random.default_rng(T + D), (T,), D, N, form, dtype)
    for k in ("x", "a", "b", "dO"):  # what lies outside every sequence must not be used
        if p[k] is not None:
            p[k][:lead] = float("nan")
            p[k][T - tail:] = float("inf")
    cud = torch.tensor(cu, device=DEV)
    keep = torch.full_like(p["x"], 7.0)
    o, h_T, ck = g.linear_forward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], o=keep, want_checkpoints=True, gates=form)
    gr = g.linear_backward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], p["dO"], p["dhT"], ck=ck, gates=form)
    torch.cuda.synchronize()
    assert (o[:lead] == 7.0).all() and (o[T - tail:] == 7.0).all()
    for k in ("dx", "da", "db"):  # no gradient reaches a row that belongs to no sequence
        if gr[k] is not None:
            assert (gr[k][:lead] == 0).all() and (gr[k][T - tail:] == 0).all(), k
    check(p, [(slice(cu[n], cu[n + 1]), n) for n in range(N)], form, o, h_T, gr)
    for n in range(N):
        if cu[n] == cu[n + 1]:
            assert torch.equal(h_T[n], p["h0"][n]) and torch.equal(gr["dh0"][n], p["dhT"][n])
    again = g.linear_backward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], p["dO"], p["dhT"], gates=form)
    for k in ("dx", "da", "db"):
        if gr[k] is not None:
            assert torch.equal(gr[k], again[k]), k
    # no initial states, no gradients of the last ones
    z = dict(p, h0=torch.zeros_like(p["h0"]), dhT=torch.zeros_like(p["dhT"]))
    o, h_T = g.linear_forward_varlen(p["x"], p["a"], p["b"], cud, gates=form)
    gr = g.linear_backward_varlen(p["x"], p["a"], p["b"], cud, None, p["dO"], gates=form)
    torch.cuda.synchronize()
    check(z, [(slice(cu[n], cu[n + 1]), n) for n in range(N)], form, o, h_T, gr)
    # states in place
    h, d = p["h0"].clone(), p["dhT"].clone()
    T2 = g.linear_forward_varlen(p["x"], p["a"], p["b"], cud, h, h_T=h, gates=form)[1]
    g2 = g.linear_backward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], p["dO"], d, grads={"dh0": d}, gates=form)
    torch.cuda.synchronize()
    assert T2 is h and g2["dh0"] is d
    check(p, [(slice(cu[n], cu[n + 1]), n) for n in range(N)], form, keep, h, dict(again, dh0=d))


@pytest.mark.parametrize("form,dtype", [("preact", "bf16"), ("channel", "f32")])
def test_more_workgroups_than_run_at_once(form, dtype):
    """13 tiles, the last one short, of 168 chains, 25 of 84: batched and packed."""
    T, D = 64 * 12 + 5, 128 * 83 + 60
    p = problem(np.random.default_rng(79), (2, T), D, 2, form, dtype)
    o, h_T, ck = g.linear_forward(p["x"], p["a"], p["b"], p["h0"], want_checkpoints=True, gates=form)
    gr = g.linear_backward(p["x"], p["a"], p["b"], p["h0"], p["dO"], p["dhT"], ck=ck, gates=form)
    torch.cuda.synchronize()
    check(p, [(0, 0), (1, 1)], form, o, h_T, gr)
    del o, ck, gr
    cu = [0, 3, 700, 700, 2 * T]  # the same tokens as three sequences and an empty one: 25 tiles
    q = dict({k: None if p[k] is None else p[k].flatten(0, 1) for k in ("x", "a", "b", "dO")},
             h0=p["h0"].repeat(2, 1), dhT=p["dhT"].repeat(2, 1))
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, h_T = g.linear_forward_varlen(q["x"], q["a"], q["b"], cud, q["h0"], gates=form)
    gr = g.linear_backward_varlen(q["x"], q["a"], q["b"], cud, q["h0"], q["dO"], q["dhT"], gates=form)
    torch.cuda.synchronize()
    check(q, [(slice(cu[n], cu[n + 1]), n) for n in range(4)], form, o, h_T, gr)


@pytest.mark.parametrize("cu", [[70], [200, 200], [0, 0, 0]])
def test_packed_tokens_of_no_sequence(cu):
    """No sequence, or empty ones only: outputs left as they were, gradients zero, states passed through."""
    f = dict(device=DEV, dtype=torch.float32)
    x, n = torch.full((200, 12), float("nan"), **f), len(cu) - 1
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    h0, dhT = torch.randn(n, 12, **f), torch.randn(n, 12, **f)
    o, h_T = g.linear_forward_varlen(x, x, x, cud, h0, o=torch.full_like(x, 7.0))
    gr = g.linear_backward_varlen(x, x, x, cud, h0, x, dhT)
    torch.cuda.synchronize()
    assert (o == 7.0).all() and torch.equal(h_T, h0) and torch.equal(gr["dh0"], dhT)
    assert all((gr[k] == 0).all() for k in ("dx", "da", "db"))


@pytest.mark.parametrize("D", [5, 64])
def test_a_bad_sequence_stays_alone(D):
    """NaN and infinities of one packed sequence reach no other one, forward and backward."""
    lens = [100, 90, 200, 10]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    p = problem(np.random.default_rng(3), (400,), D, 4, "channel", "f32")
    for at, v in ((120, float("nan")), (130, float("inf"))):
        p["x"][at] = v
        p["dO"][at] = v
    cud = torch.tensor(cu, device=DEV)
    o, h_T, ck = g.linear_forward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], want_checkpoints=True)
    gr = g.linear_backward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], p["dO"], p["dhT"], ck=ck)
    torch.cuda.synchronize()
    assert torch.isnan(o[120:190]).all() and torch.isfinite(o[100:120]).all()
    check(p, [(slice(cu[n], cu[n + 1]), n) for n in (0, 2, 3)], "channel", o, h_T, gr)


@pytest.mark.parametrize("value", [0.0, 1.0])
def test_decays_of_zero_and_one(value):
    """a = 0 forgets at once (o = b x exactly); a = 1 is a running sum."""
    rng = np.random.default_rng(5)
    p = problem(rng, (2, 700), 12, 2, "channel", "f32")
    p["a"].fill_(value)
    o, h_T = g.linear_forward(p["x"], p["a"], p["b"], p["h0"])
    torch.cuda.synchronize()
    if value == 0.0:
        assert torch.equal(o, p["x"] * p["b"])
    for n in range(2):
        ro, _ = R.linear(R.f64(p["x"])[n], R.f64(p["a"])[n], R.f64(p["b"])[n], R.f64(p["h0"])[n], "channel")
        # 700 terms: every partial sum is off by at most one rounding of the product and one of each of 700 sums
        assert np.abs(R.f64(o[n]) - ro).max() <= 2 * 700 * R.U32 * np.abs(ro).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["preact", "tied_preact"])
def test_far_preactivations(form, dtype):
    """Pre-activations of +-100 and +-inf: decays of 1 and 0 to within 2e-38, and finite gradients."""
    T, D = 6, 4
    pre = torch.tensor([-100.0, -float("inf"), -90.0, 100.0, float("inf"), 90.0], device=DEV)
    a = pre[None, :, None].expand(1, T, D).contiguous()
    b = None if form == "tied_preact" else (-pre)[None, :, None].expand(1, T, D).contiguous()
    x = torch.ones(1, T, D, device=DEV).to(R.TORCH[dtype])
    a, b = a.to(x.dtype), None if b is None else b.to(x.dtype)
    h0 = torch.full((1, D), 3.0, device=DEV)
    o, _ = g.linear_forward(x, a, b, h0, gates=form)
    gr = g.linear_backward(x, a, b, h0, torch.ones_like(x), gates=form)
    torch.cuda.synchronize()
    # tied: the first three keep 3, then h = x = 1; with an input gate of sigmoid(-pre): 3 + 1 + 1 + 1, then 0
    want = [3, 3, 3, 1, 1, 1] if form == "tied_preact" else [4, 5, 6, 0, 0, 0]
    assert (o[0, :, 0].float().cpu() - torch.tensor(want, dtype=torch.float32)).abs().max() <= 1e-30
    assert all(torch.isfinite(v).all() for v in gr.values() if v is not None)


def test_no_tokens_and_no_sequences():
    f = dict(device=DEV, dtype=torch.float32)
    h0, dhT = torch.randn(3, 8, **f), torch.randn(3, 8, **f)
    e = torch.empty(3, 0, 8, **f)
    o, h_T = g.linear_forward(e, e, e, h0)
    gr = g.linear_backward(e, e, e, h0, e, dhT)
    torch.cuda.synchronize()
    assert o.shape == (3, 0, 8) and torch.equal(h_T, h0) and torch.equal(gr["dh0"], dhT)
    e = torch.empty(0, 5, 8, **f)
    o, h_T = g.linear_forward(e, e, e)
    assert o.shape == (0, 5, 8) and h_T.shape == (0, 8)
    gr = g.linear_backward(e, e, e, None, e)
    assert gr["dx"].shape == (0, 5, 8)
    e = torch.empty(0, 8, **f)
    o, h_T = g.linear_forward_varlen(e, e, e, torch.zeros(4, dtype=torch.int32, device=DEV), h0)
    torch.cuda.synchronize()
    assert o.shape == (0, 8) and torch.equal(h_T, h0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", R.FORMS)
@pytest.mark.parametrize("N,D", [(1, 1), (3, 7), (256, 64), (5, 2052)])
def test_step_continues_a_prefill(N, D, form, dtype):
    p = problem(np.random.default_rng(N + D), (N, 4), D, N, form, dtype)
    h = p["h0"].clone()
    cols = []
    for t in range(4):
        at = lambda v: None if v is None else v[:, t].contiguous()
        if t % 2:
            out = torch.full_like(h, float("nan"))
            cols.append(g.linear_step(at(p["x"]), at(p["a"]), at(p["b"]), h, h_out=out, gates=form))
            h = out
        else:
            cols.append(g.linear_step(at(p["x"]), at(p["a"]), at(p["b"]), h, gates=form))
    o = torch.stack(cols, 1)
    torch.cuda.synchronize()
    check(p, [(n, n) for n in range(0, N, max(1, N // 5))], form, o, h)


def test_in_place_states_and_repeatability():
    p = problem(np.random.default_rng(11), (2, 900), 70, 2, "preact", "bf16")
    o1, T1, ck = g.linear_forward(p["x"], p["a"], p["b"], p["h0"], want_checkpoints=True, gates="preact")
    h = p["h0"].clone()
    o2, T2 = g.linear_forward(p["x"], p["a"], p["b"], h, h_T=h, gates="preact")
    g1 = g.linear_backward(p["x"], p["a"], p["b"], p["h0"], p["dO"], p["dhT"], ck=ck, gates="preact")
    d = p["dhT"].clone()
    g2 = g.linear_backward(p["x"], p["a"], p["b"], p["h0"], p["dO"], d, ck=ck, grads={"dh0": d}, gates="preact")
    torch.cuda.synchronize()
    assert T2 is h and torch.equal(o1, o2) and torch.equal(T1, T2)
    assert g2["dh0"] is d and all(torch.equal(g1[k], g2[k]) for k in g1)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("form", R.FORMS)
def test_gradients_against_differences(form, packed):
    """The gradient along a random direction against central differences of the
    64-bit plain form. The difference's own error is step^2 times a third
    derivative (1e-10 times values of order 1e3 here) and 1e-16 / 1e-5 of the loss."""
    rng = np.random.default_rng(17)
    lens, D = ([60, 0, 140], 6) if packed else ([200], 6)
    cu = np.concatenate([[0], np.cumsum(lens)])
    p = problem(rng, (200,), D, len(lens), form, "f32")
    leaf = {k: p[k].clone().requires_grad_() for k in ("x", "a", "b", "h0") if p[k] is not None}
    if packed:
        o, h_T = g.gated_linear_recurrence_varlen(leaf["x"], leaf["a"], leaf.get("b"),
                                                  torch.tensor(cu, dtype=torch.int32, device=DEV), leaf["h0"], gates=form)
    else:
        one = lambda k: None if k not in leaf else leaf[k][None]
        o, h_T = g.gated_linear_recurrence(one("x"), one("a"), one("b"), leaf["h0"], gates=form)
        o = o[0]
    grads = dict(zip(leaf, torch.autograd.grad((o, h_T), list(leaf.values()), (p["dO"], p["dhT"]))))
    f = {k: R.f64(v) for k, v in p.items()}

    def loss(q):
        s = 0.0
        for n in range(len(lens)):
            at = slice(cu[n], cu[n + 1])
            ro, rT = R.linear(q["x"][at], q["a"][at], None if q["b"] is None else q["b"][at], q["h0"][n], form)
            s += (ro * f["dO"][at]).sum() + (rT * f["dhT"][n]).sum()
        return s

    for k in leaf:
        v = rng.standard_normal(f[k].shape)
        step = 1e-5
        up, dn = dict(f, **{k: f[k] + step * v}), dict(f, **{k: f[k] - step * v})
        num = (loss(up) - loss(dn)) / (2 * step)
        terms = R.f64(grads[k]) * v
        scale = np.abs(R.f64(grads[k])).max() * np.abs(v).sum()
        print(f"[linear differences {form} {k}] {terms.sum():.8g} {num:.8g}", flush=True)
        assert abs(terms.sum() - num) <= 2 * E32 * scale + 1e-6 * (1 + abs(num))


def test_another_stream_and_a_replayed_graph():
    p = problem(np.random.default_rng(23), (1, 3000), 64, 1, "channel", "bf16")
    args = (p["x"], p["a"], p["b"], p["h0"])
    o, h_T, ck = g.linear_forward(*args, want_checkpoints=True)
    gr = g.linear_backward(*args, p["dO"], p["dhT"], ck=ck)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, T2 = g.linear_forward(*args, stream=s)
    o3, T3 = g.linear_forward(*args, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(h_T, T2) and torch.equal(o, o3) and torch.equal(h_T, T3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o4, T4, ck4 = g.linear_forward(*args, want_checkpoints=True)
        g4 = g.linear_backward(*args, p["dO"], p["dhT"], ck=ck4)
    for i in range(4):
        for t in (o4, T4, g4["dx"], g4["da"], g4["db"], g4["dh0"]):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o4) and torch.equal(h_T, T4), i
        assert all(torch.equal(gr[k], g4[k]) for k in gr), i
        o2, _ = g.linear_forward(*args)  # eager work of its own between the replays
        torch.cuda.synchronize()
        assert torch.equal(o, o2), i


def test_offsets_past_32_bits():
    """2^31 + values in x, o and the gates: the last sequence and a middle token against the plain form."""
    D, T = 4096, 1 << 18
    B = 2  # 2^31 elements, 4 GiB a bf16 tensor; the second sequence starts at byte 2^31 and ends at 2^32
    x = torch.zeros(B, T, D, dtype=torch.bfloat16, device=DEV)
    a = torch.full((B, T, D), 2.0, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(29)
    cols = [0, 63, 64, 2049, 4095]
    last = 300  # with decays of at most 0.2 older tokens weigh less than 0.2^300
    xs, as_ = rng.standard_normal((last, 5)), rng.uniform(1.4, 3.0, (last, 5))
    x[1, T - last:, cols] = torch.tensor(xs, dtype=torch.bfloat16, device=DEV)
    a[1, T - last:, cols] = torch.tensor(as_, dtype=torch.bfloat16, device=DEV)
    o, h_T = g.linear_forward(x, a, gates="tied_preact")
    torch.cuda.synchronize()
    ro, rT = R.linear(R.f64(x[1, T - last:, cols]), R.f64(a[1, T - last:, cols]), None, np.zeros(5), "tied_preact")
    close("o", o[1, T - last:, cols], ro, np.abs(ro).max(), torch.bfloat16)
    close("h_T", h_T[1, cols], rT, np.abs(ro).max())
    assert (o[0] == 0).all()
    del o
    # the gradients of the last tokens: what lies before them weighs less than 0.2^250
    dO = torch.zeros_like(x)
    dO[1, T - 50:, cols] = x[1, T - 50:, cols]
    gr = g.linear_backward(x, a, None, None, dO, gates="tied_preact")
    torch.cuda.synchronize()
    sl = (1, slice(T - last, None), cols)
    dx, da, _, _, ad = R.linear_grads(R.f64(x[sl]), R.f64(a[sl]), None, np.zeros(5), R.f64(dO[sl]), np.zeros(5), "tied_preact")
    close("dx", gr["dx"][sl], dx, np.abs(ad).max(), torch.bfloat16)
    close("da", gr["da"][sl], da, np.abs(ad).max() * 2 * np.abs(R.f64(x[sl])).max(), torch.bfloat16, 2.0)
    assert (gr["dx"][0] == 0).all()


def test_more_sequences_than_workgroups():
    """6000 sequences of 0 to 5 tokens at a width where each has 32 blocks of channels: batches of single tokens and
    short prompts as a server packs them."""
    rng = np.random.default_rng(31)
    lens = rng.integers(0, 6, 6000)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, D, N = int(cu[-1]), 4096, 6000
    p = problem(rng, (T,), D, N, "preact", "bf16")
    cud = torch.tensor(cu, device=DEV)
    o, h_T, ck = g.linear_forward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], want_checkpoints=True, gates="preact")
    gr = g.linear_backward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], p["dO"], p["dhT"], ck=ck, gates="preact")
    torch.cuda.synchronize()
    some = [0, 1, 2, 3000, 3001, 5998, 5999] + list(np.argwhere(lens == 0)[:5, 0]) + list(rng.integers(0, N, 20))
    check(p, [(slice(cu[n], cu[n + 1]), n) for n in some], "preact", o, h_T, gr)
    empty = torch.tensor(lens == 0, device=DEV)
    assert torch.equal(h_T[empty], p["h0"][empty]) and torch.equal(gr["dh0"][empty], p["dhT"][empty])


@pytest.mark.parametrize("N,T", [(4096, 64), (4096, 130), (4096, 0)])
def test_states_of_empty_sequences_pass_through_by_the_whole_card(N, T):
    """A few tokens among thousands of empty sequences: 64 MiB of states are passed on, in at most ten times a copy's
    time and 100 us (one workgroup would take hundreds of times it), forward and backward."""
    D = 4096
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[N // 2:] = T  # all tokens in one sequence
    cu = cu.to(DEV)
    p = problem(np.random.default_rng(37), (max(T, 1),), D, 1, "channel", "f32")
    x, a, b, dO = (p[k][:T] for k in ("x", "a", "b", "dO"))
    h0 = torch.randn(N, D, device=DEV)
    h_T = torch.empty_like(h0)

    def us(f):
        times = []
        for _ in range(6):
            s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            s.record()
            f()
            e.record()
            e.synchronize()
            times.append(s.elapsed_time(e) * 1e3)
        return min(times[1:])

    copy = us(lambda: h_T.copy_(h0))
    fwd = us(lambda: g.linear_forward_varlen(x, a, b, cu, h0, h_T=h_T))
    gr = {"dh0": torch.empty_like(h0)}
    bwd = us(lambda: g.linear_backward_varlen(x, a, b, cu, h0, dO, h_T, grads=gr))
    print(f"[linear empty sequences T {T}] copy {copy:.0f} us, forward {fwd:.0f}, backward {bwd:.0f}", flush=True)
    rest = torch.arange(N, device=DEV) != (N // 2 - 1 if T else -1)
    assert torch.equal(h_T[rest], h0[rest]) and torch.equal(gr["dh0"][rest], h_T[rest])
    assert fwd <= 10 * copy + 100 and bwd <= 10 * copy + 100


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("value", [0.05, 0.0])
@pytest.mark.parametrize("D", [5, 64])
def test_a_bad_token_reaches_its_sequences_end(D, value, packed):
    """With decays whose product over a tile is 0 in fp32 (and with decays of 0: 0 * NaN is NaN) a NaN still reaches
    every later token of its sequence, and in the backward every earlier one, but no other sequence."""
    cu, n = [0, 30, 730, 900], 1
    p = problem(np.random.default_rng(41), (900,), D, 3, "channel", "f32")
    p["a"].fill_(value)
    p["x"][100], p["dO"][650] = float("nan"), float("nan")
    if packed:
        cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
        o, h_T, ck = g.linear_forward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], want_checkpoints=True)
        gr = g.linear_backward_varlen(p["x"], p["a"], p["b"], cud, p["h0"], p["dO"], p["dhT"], ck=ck)
    else:
        q = {k: p[k][None, 30:730] for k in ("x", "a", "b", "dO")}
        o, h_T, ck = g.linear_forward(q["x"], q["a"], q["b"], p["h0"][1:2], want_checkpoints=True)
        gr = g.linear_backward(q["x"], q["a"], q["b"], p["h0"][1:2], q["dO"], p["dhT"][1:2], ck=ck)
        o, gr, cu, n = o[0], {k: v[0] if k != "dh0" else v for k, v in gr.items()}, [0, 700], 0
    torch.cuda.synchronize()
    lo, hi, bad, badO = cu[n], cu[n + 1], cu[n] + 70, cu[n] + 620
    assert torch.isnan(o[bad:hi]).all() and torch.isnan(h_T[n]).all() and torch.isfinite(o[lo:bad]).all()
    assert torch.isnan(gr["dx"][lo:badO + 1]).all() and torch.isnan(gr["dh0"][n]).all()
    assert torch.isfinite(gr["dx"][badO + 1:hi]).all() and torch.isnan(gr["da"][bad + 1:hi]).all()
    if packed:
        p = dict(p, x=p["x"].nan_to_num(0.0), dO=p["dO"].nan_to_num(0.0))
        check(p, [(slice(cu[m], cu[m + 1]), m) for m in (0, 2)], "channel", o, h_T, gr)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["preact", "tied_preact"])
@pytest.mark.parametrize("T,D,packed", [(1, 64, False), (1, 61, False), (128, 64, False), (128, 61, False), (128, 64, True)])
def test_gradients_of_nearly_closed_and_open_gates(T, D, packed, form, dtype):
    """Value by value: pre-activations of +-8 to +-20, where one of a gate and its complement is 2e-9 to 3e-4. States,
    adjoints and terms are all of one sign, so nothing cancels and each gradient is held to its own size: T tokens'
    30 roundings (20 of them the exponential's argument's) for each of the state and the adjoint, 60 of the two
    factors, and the output's one."""
    rng = np.random.default_rng(43)
    mk = lambda v, d: torch.tensor(np.asarray(v, np.float32)).to(d).to(DEV)
    dt, shape = R.TORCH[dtype], (1, T, D)
    far = np.linspace(8.0, 20.0, D) * np.where(np.arange(D) % 2, 1.0, -1.0)
    # tied: h - x must not cancel, so x changes its sign from token to token (a closed gate's h is the x before)
    sign = np.where(np.arange(T) % 2, -1.0, 1.0)[None, :, None] if form == "tied_preact" else 1.0
    x, dO = sign * rng.uniform(0.5, 1.5, shape), rng.uniform(0.5, 1.5, shape)
    a = np.ascontiguousarray(np.broadcast_to(far, shape))
    b = np.ascontiguousarray(np.broadcast_to(np.roll(far, D // 2), shape))
    h0, dhT = np.full((1, D), -3.0 if form == "tied_preact" else 3.0), np.full((1, D), 2.0)
    p = dict(x=mk(x, dt), a=mk(a, dt), b=None if form == "tied_preact" else mk(b, dt), h0=mk(h0, torch.float32),
             dO=mk(dO, dt), dhT=mk(dhT, torch.float32))
    if packed:
        q = {k: None if p[k] is None else p[k][0] for k in ("x", "a", "b", "dO")}
        cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
        gr = g.linear_backward_varlen(q["x"], q["a"], q["b"], cu, p["h0"], q["dO"], p["dhT"], gates=form)
    else:
        gr = g.linear_backward(p["x"], p["a"], p["b"], p["h0"], p["dO"], p["dhT"], gates=form)
    torch.cuda.synchronize()
    f = {k: R.f64(v) for k, v in p.items()}
    one = lambda k: None if f[k] is None else f[k][0]
    dx, da, db, dh0, _ = R.linear_grads(f["x"][0], f["a"][0], one("b"), f["h0"][0], f["dO"][0], f["dhT"][0], form)
    rel = (60 * T + 60) * R.U32
    for name, got, ref, r in (("da", gr["da"], da, rel), ("db", gr["db"], db, rel), ("dx", gr["dx"], dx, rel), ("dh0", gr["dh0"], dh0, rel)):
        if ref is None:
            continue
        r = r + (0.0 if got.dtype == torch.float32 else R.half(got.dtype) * (1 + r))
        worst = (np.abs(R.f64(got).reshape(ref.shape) - ref) / (r * np.abs(ref))).max()
        print(f"[linear gates {form} {dtype} T {T} {name}] worst error over its bound {worst:.3f}", flush=True)
        assert worst <= 1.0, name
