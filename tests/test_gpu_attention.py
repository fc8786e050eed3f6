"""Softmax attention (gdn2_attention_*) against its 64-bit plain form; the bounds
are derived in attention_ref."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rand(rng, *shape, dtype="bf16", std=1.0):
    return torch.tensor((std * rng.standard_normal(shape)).astype(np.float32)).to(R.TYPES[dtype]).to(DEV)


def problem(seed, B, T, S, H, Hkv, d, dtype):
    rng = np.random.default_rng(seed)
    return (rand(rng, B, T, H, d, dtype=dtype), rand(rng, B, S, Hkv, d, dtype=dtype), rand(rng, B, S, Hkv, d, dtype=dtype),
            rand(rng, B, T, H, d, dtype=dtype))


def check(name, q, k, v, dO, o, lse, gr, causal=True, window=0, scale=None):
    """One batch, sequence by sequence."""
    scale = float(np.float32(q.shape[-1] ** -0.5 if scale is None else scale))
    for b in range(q.shape[0]):
        ref = R.grouped(q[b], k[b], v[b], None if gr is None else dO[b], scale, causal, window, q.dtype)
        got = {"o": o[b], "lse": lse[b]}
        if gr is not None:
            got.update(dq=gr["dq"][b], dk=gr["dk"][b], dv=gr["dv"][b])
        for n, (x, t) in ref.items():
            R.hold(f"{name} {n}", got[n], x, t)


def run(q, k, v, dO, **kw):
    o, lse = g.attention_forward(q, k, v, **kw)
    gr = None if dO is None else g.attention_backward(q, k, v, o, lse, dO, **kw)
    torch.cuda.synchronize()
    return o, lse, gr


# (T, S, causal, window): one token to several blocks, around the edges of tiles and blocks, prefixes, queries without keys
SIZES = [(1, 1, True, 0), (1, 1, False, 0), (2, 2, True, 0), (31, 31, True, 0), (33, 33, True, 0), (64, 64, True, 0),
         (65, 65, True, 0), (127, 127, True, 0), (128, 128, True, 0), (129, 129, True, 0), (257, 257, True, 0),
         (300, 300, False, 0), (1, 200, True, 0), (1, 200, False, 0), (70, 333, True, 0), (200, 65, False, 0),
         (90, 40, True, 0), (300, 100, True, 0), (1, 500, True, 7), (200, 200, True, 1), (200, 200, True, 33),
         (333, 333, True, 64), (300, 300, True, 128), (150, 400, True, 100), (400, 150, True, 60), (40, 90, True, 1000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,S,causal,window", SIZES)
def test_forward_and_gradients(T, S, causal, window, d, dtype):
    B, H, Hkv = 2, 4, 2
    q, k, v, dO = problem(T * 7 + S + window, B, T, S, H, Hkv, d, dtype)
    o, lse, gr = run(q, k, v, dO, causal=causal, window=window)
    check(f"attention {T} {S} {causal} {window} d{d} {dtype}", q, k, v, dO, o, lse, gr, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 1), (6, 3), (8, 1), (3, 3), (16, 2)])
def test_head_layouts(H, Hkv, dtype):
    q, k, v, dO = problem(H * 10 + Hkv, 1, 150, 170, H, Hkv, 64, dtype)
    o, lse, gr = run(q, k, v, dO)
    check(f"attention heads {H}/{Hkv} {dtype}", q, k, v, dO, o, lse, gr)


@pytest.mark.parametrize("d,H,Hkv,T,window,causal", [(128, 48, 4, 300, 0, True), (128, 64, 2, 260, 0, False),
                                                      (64, 96, 16, 290, 50, True), (128, 120, 20, 640, 100, True)])
def test_many_heads(d, H, Hkv, T, window, causal):
    """Enough workgroups for key blocks of 128 rows, and for fewer parts than a key head has query heads."""
    q, k, v, dO = problem(H + T, 1 if T > 300 else 2, T, T, H, Hkv, d, "bf16")
    o, lse, gr = run(q, k, v, dO, window=window, causal=causal)
    check(f"attention heads {H}/{Hkv} d{d} {window} {causal}", q, k, v, dO, o, lse, gr, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,window,causal", [(64, 0, True), (128, 0, True), (64, 90, True), (128, 0, False)])
def test_more_blocks_than_run_at_once(d, window, causal, dtype):
    q, k, v, dO = problem(d + window, 4, 131, 140, 72, 36, d, dtype)
    o, lse, gr = run(q, k, v, dO, window=window, causal=causal)
    check(f"attention blocks d{d} {window} {causal} {dtype}", q, k, v, dO, o, lse, gr, causal, window)


def test_many_heads_of_packed_sequences():
    lengths = [140, 0, 128, 1, 200, 60]
    q, k, v, dO, cu, _ = packed(12, lengths, lengths, 56, 4, 128, "bf16", front=2, behind=5)
    o, lse = g.attention_forward_varlen(q, k, v, cu)
    gr = g.attention_backward_varlen(q, k, v, o, lse, dO, cu)
    torch.cuda.synchronize()
    check_packed("packed, many heads", q, k, v, dO, cu, cu, o, lse, gr)


LENGTHS = [[5], [0, 0, 3, 0], [128, 1, 127, 129, 0, 64], [300, 0, 1, 33, 250], [1] * 70, [0] * 5]


def packed(seed, lq, lk, H, Hkv, d, dtype, front=0, behind=0):
    rng = np.random.default_rng(seed)
    off = lambda ls: torch.tensor(np.concatenate(([0], np.cumsum(ls))) + front, dtype=torch.int32, device=DEV)  # noqa: E731
    T, S = sum(lq) + front + behind, sum(lk) + front + behind
    return (rand(rng, T, H, d, dtype=dtype), rand(rng, S, Hkv, d, dtype=dtype), rand(rng, S, Hkv, d, dtype=dtype),
            rand(rng, T, H, d, dtype=dtype), off(lq), off(lk))


def check_packed(name, q, k, v, dO, cu_q, cu_k, o, lse, gr, window=0, causal=True):
    scale = float(np.float32(q.shape[-1] ** -0.5))
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for n in range(len(cq) - 1):
        a, c = slice(cq[n], cq[n + 1]), slice(ck[n], ck[n + 1])
        ref = R.grouped(q[a], k[c], v[c], dO[a], scale, causal, window, q.dtype)
        got = dict(o=o[a], lse=lse[:, a], dq=gr["dq"][a], dk=gr["dk"][c], dv=gr["dv"][c])
        for nm, (x, t) in ref.items():
            R.hold(f"{name} sequence {n} {nm}", got[nm], x, t)
    for nm, cu in (("dq", cq), ("dk", ck), ("dv", ck)):
        assert (gr[nm][:cu[0]] == 0).all() and (gr[nm][cu[-1]:] == 0).all(), nm


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_packed_sequences(lengths, window, dtype):
    q, k, v, dO, cu, _ = packed(sum(lengths), lengths, lengths, 4, 2, 64, dtype, front=3, behind=70)
    o, lse = torch.full_like(q, 7.0), torch.full((4, q.shape[0]), 7.0, device=DEV)
    g.attention_forward_varlen(q, k, v, cu, window=window, o=o, lse=lse)
    gr = g.attention_backward_varlen(q, k, v, o, lse, dO, cu, window=window)
    torch.cuda.synchronize()
    check_packed(f"packed {dtype}", q, k, v, dO, cu, cu, o, lse, gr, window)
    for x in (o, lse.T):  # rows of no sequence are left as they were
        assert (x[:3] == 7.0).all() and (x[int(cu[-1]):] == 7.0).all()


@pytest.mark.parametrize("causal", [True, False])
def test_packed_queries_behind_prefixes(causal):
    """Each sequence with keys of its own number: more than its queries, as many, fewer, none."""
    lq, lk = [10, 1, 130, 20, 0, 7, 40], [200, 77, 130, 5, 9, 0, 41]
    q, k, v, dO, cu_q, cu_k = packed(3, lq, lk, 6, 2, 128, "bf16")
    o, lse = g.attention_forward_varlen(q, k, v, cu_q, cu_k, causal=causal)
    gr = g.attention_backward_varlen(q, k, v, o, lse, dO, cu_q, cu_k, causal=causal)
    torch.cuda.synchronize()
    check_packed(f"prefixes {causal}", q, k, v, dO, cu_q, cu_k, o, lse, gr, causal=causal)


def test_a_packed_sequence_is_the_sequence_alone():
    q, k, v, dO, cu, _ = packed(5, [100, 333, 64], [100, 333, 64], 8, 2, 128, "bf16")
    o, lse = g.attention_forward_varlen(q, k, v, cu)
    c = cu.tolist()
    for a, b in zip(c, c[1:]):
        o1, l1 = g.attention_forward(q[None, a:b], k[None, a:b], v[None, a:b])
        torch.cuda.synchronize()
        assert torch.equal(o[a:b], o1[0]) and torch.equal(lse[:, a:b], l1[0])


@pytest.mark.parametrize("T,S", [(5, 0), (0, 5), (200, 0), (0, 200)])
def test_no_keys_or_no_queries(T, S):
    q, k, v, dO = problem(T + S, 2, T, S, 4, 2, 64, "bf16")
    o, lse, gr = run(q, k, v, dO)
    assert (o == 0).all() and (lse == -float("inf")).all()
    assert all((x == 0).all() and x.shape == t.shape for x, t in zip(gr.values(), (q, k, v)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_query_that_is_no_number(dtype):
    q, k, v, dO = problem(8, 1, 150, 150, 2, 1, 64, dtype)
    q[0, 70, 1, 5] = float("nan")
    o, lse, gr = run(q, k, v, dO)
    assert torch.isnan(o[0, 70, 1]).all() and torch.isnan(lse[0, 1, 70])
    o[0, 70, 1], lse[0, 1, 70] = 0, 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert torch.isnan(gr["dq"][0, 70, 1]).all() and torch.isfinite(gr["dq"][0, 70, 0]).all()
    for nm in ("dk", "dv"):  # the keys that it sees
        assert torch.isnan(gr[nm][0, :71]).all() and torch.isfinite(gr[nm][0, 71:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hidden_values_in_more_blocks_than_run_at_once(dtype):
    """Infinities and NaN that no query sees, and one that later queries see."""
    q, k, v, _ = problem(9, 4, 200, 200, 72, 72, 64, dtype)
    o, lse = g.attention_forward(q, k, v)
    k[:, 150, :, 1], v[:, 151, :, 2], v[:, 199, :, 3] = float("nan"), float("inf"), -float("inf")
    o2, lse2 = g.attention_forward(q, k, v)
    torch.cuda.synchronize()
    assert torch.equal(o[:, :150], o2[:, :150]) and torch.equal(lse[:, :, :150], lse2[:, :, :150])
    assert torch.isnan(o2[:, 150:]).all() and torch.isnan(lse2[:, :, 150:]).all()
    k[:, 150, :, 1] = 0
    o2, _ = g.attention_forward(q, k, v)
    torch.cuda.synchronize()
    assert torch.isfinite(o2[:, :151]).all() and not torch.isfinite(o2[:, 151:, :, 2]).any()
    assert torch.isfinite(o2[:, :199, :, 3]).all() and torch.isfinite(o2[:, :, :, 4:]).all()


def test_offsets_outside_the_tokens_are_clamped():
    q, k, v, dO, _, _ = packed(6, [200], [200], 2, 1, 64, "bf16")
    far = torch.tensor([-50, 120, 10 ** 9], dtype=torch.int32, device=DEV)
    near = torch.tensor([0, 120, 200], dtype=torch.int32, device=DEV)
    res = []
    for cu in (far, near):
        o, lse = g.attention_forward_varlen(q, k, v, cu)
        res.append((o, lse, *g.attention_backward_varlen(q, k, v, o, lse, dO, cu).values()))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*res))


def test_many_packed_sequences():
    """Enough that the search for a block's sequence takes three rounds."""
    rng = np.random.default_rng(9)
    lengths = rng.integers(0, 3, 5000).tolist()
    lengths[4321] = 300
    q, k, v, dO, cu, _ = packed(9, lengths, lengths, 1, 1, 64, "bf16")
    o, lse = g.attention_forward_varlen(q, k, v, cu)
    gr = g.attention_backward_varlen(q, k, v, o, lse, dO, cu)
    torch.cuda.synchronize()
    c = cu.tolist()
    for n in (0, 1, 63, 64, 65, 4095, 4096, 4320, 4321, 4322, 4999):
        a, b = c[n], c[n + 1]
        ref = R.grouped(q[a:b], k[a:b], v[a:b], dO[a:b], float(np.float32(0.125)), True, 0, q.dtype)
        for nm, got in (("o", o), ("dq", gr["dq"]), ("dk", gr["dk"]), ("dv", gr["dv"])):
            R.hold(f"many {n} {nm}", got[a:b], *ref[nm])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_parts_of_a_fused_projection(dtype):
    B, T, H, Hkv, d = 2, 140, 4, 2, 64
    rng = np.random.default_rng(11)
    qkv = rand(rng, B, T, (H + 2 * Hkv) * d, dtype=dtype)
    parts = [x.unflatten(-1, (-1, d)) for x in qkv.split([H * d, Hkv * d, Hkv * d], -1)]
    dO = rand(rng, B, T, H, d, dtype=dtype)
    o, lse, gr = run(*parts, dO)
    o2, lse2, gr2 = run(*[x.contiguous() for x in parts], dO)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(gr[n], gr2[n]) for n in gr)
    # through autograd, to the projection itself
    leaf = qkv.detach().requires_grad_()
    parts = [x.unflatten(-1, (-1, d)) for x in leaf.split([H * d, Hkv * d, Hkv * d], -1)]
    got, = torch.autograd.grad(g.attention(*parts), leaf, dO)
    want = torch.cat([gr[n].flatten(-2) for n in ("dq", "dk", "dv")], -1)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("place", [70, 127, 128, 199])
def test_hidden_values_leave_nothing(place, bad, dtype):
    """Values that are no number in one key: rows that do not see it are what they are without it, to the bit; rows
    that do see it become NaN."""
    B, T, H, Hkv, d = 1, 200, 2, 1, 64
    q, k, v, dO = problem(place, B, T, T, H, Hkv, d, dtype)
    o, lse, gr = run(q, k, v, dO, window=50)
    for which in ("v", "k"):
        k2, v2 = k.clone(), v.clone()
        (v2 if which == "v" else k2)[0, place, 0, 5] = bad
        o2, lse2, gr2 = run(q, k2, v2, dO, window=50)
        free = [i for i in range(T) if i < place or i >= place + 50]
        seen = [i for i in range(place, min(T, place + 50))]
        assert torch.equal(o[:, free], o2[:, free]) and torch.equal(lse[:, :, free], lse2[:, :, free]), which
        assert torch.equal(gr["dq"][:, free], gr2["dq"][:, free]), which
        if which == "v":  # its own channel alone, and the softmax not at all
            assert not torch.isfinite(o2[:, seen][..., 5]).any() and torch.equal(lse, lse2)
            assert torch.equal(o[..., :5], o2[..., :5]) and torch.equal(o[..., 6:], o2[..., 6:])
        elif np.isnan(bad):
            assert torch.isnan(o2[:, seen]).all() and torch.isnan(lse2[:, :, seen]).all()
        # keys that share no query with it
        far = [j for j in range(T) if j < place - 49 or j >= place + 50]
        assert torch.equal(gr["dk"][:, far], gr2["dk"][:, far]) and torch.equal(gr["dv"][:, far], gr2["dv"][:, far])
    # and in one query: only its own row, and the keys that it sees
    q2, dO2 = q.clone(), dO.clone()
    q2[0, place, 0, 3] = bad
    o2, lse2, gr2 = run(q2, k, v, dO, window=50)
    rest = [i for i in range(T) if i != place]
    unseen = [j for j in range(T) if j > place or j <= place - 50]
    assert torch.equal(o[:, rest], o2[:, rest]) and torch.equal(gr["dq"][:, rest], gr2["dq"][:, rest])
    assert torch.equal(gr["dk"][:, unseen], gr2["dk"][:, unseen]) and torch.equal(gr["dv"][:, unseen], gr2["dv"][:, unseen])
    dO2[0, place, 1, 9] = bad
    gr2 = g.attention_backward(q, k, v, o, lse, dO2, window=50)
    torch.cuda.synchronize()
    assert torch.equal(gr["dk"][:, unseen], gr2["dk"][:, unseen]) and torch.equal(gr["dv"][:, unseen], gr2["dv"][:, unseen])
    saw = [j for j in range(max(0, place - 49), place + 1)]
    assert not torch.isfinite(gr2["dv"][:, saw][..., 9]).any() and torch.isfinite(gr2["dv"][..., :9]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_behind_the_prompts(dtype):
    """A batch padded at the end with NaN: causal rows before it do not see it."""
    q, k, v, dO = problem(21, 2, 190, 190, 4, 4, 128, dtype)
    o, lse, _ = run(q, k, v, None)
    for x in (q, k, v):
        x[0, 101:] = float("nan")
        x[1, 64:] = float("inf")
    o2, lse2, _ = run(q, k, v, None)
    assert torch.equal(o[0, :101], o2[0, :101]) and torch.equal(o[1, :64], o2[1, :64])
    assert torch.equal(lse[0, :, :101], lse2[0, :, :101]) and torch.equal(lse[1, :, :64], lse2[1, :, :64])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Scores of several hundred, one key far above the rest in every row, and rows whose scores fall by hundreds from
    one tile to the next."""
    q, k, v, dO = problem(31, 1, 260, 260, 2, 1, 64, dtype)
    k[0, ::61] *= 30
    k[0, :64] *= 20
    scale = 0.5
    o, lse, gr = run(q, k, v, dO, scale=scale)
    for b in range(1):
        ref = R.grouped(q[b], k[b], v[b], None, scale, True, 0, q.dtype)
        for n, x in (("o", o[b]), ("lse", lse[b])):
            R.hold(f"large scores {n} {dtype}", x, *ref[n])
    assert all(torch.isfinite(x).all() for x in gr.values())


@pytest.mark.parametrize("d,window,causal", [(64, 0, True), (128, 9, True), (64, 0, False)])
def test_gradients_against_differences(d, window, causal):
    """Along random directions against central differences of the 64-bit plain form."""
    q, k, v, dO = problem(41, 1, 40, 50, 4, 2, d, "f32")
    scale = float(np.float32(d ** -0.5))
    leaf = [x.clone().requires_grad_() for x in (q, k, v)]
    grads = torch.autograd.grad(g.attention(*leaf, causal=causal, window=window), leaf, dO)
    f = [R.f64(x) for x in (q, k, v)]
    G = R.f64(dO)[0]

    def loss(parts):
        total = 0.0
        for h in range(4):
            r = R.attention(parts[0][0][:, h], parts[1][0][:, h // 2], parts[2][0][:, h // 2], None, scale, causal, window, q.dtype)
            total += (r["o"][0] * G[:, h]).sum()
        return total

    rng = np.random.default_rng(42)
    for i, nm in enumerate("qkv"):
        w = rng.standard_normal(f[i].shape)
        step = lambda e: loss([x + e * w if j == i else x for j, x in enumerate(f)])  # noqa: E731, B023
        num, got = (step(1e-5) - step(-1e-5)) / 2e-5, (R.f64(grads[i]) * w).sum()
        print(f"[attention differences {nm}] {got:.8g} {num:.8g}", flush=True)
        # at most 256 roundings of each gradient value, and the differences' own error
        assert abs(got - num) <= 256 * R.U * np.abs(R.f64(grads[i])).max() * np.abs(w).sum() + 1e-6 * (1 + abs(num))


def test_replayed_graphs_repeatability_and_a_shared_workspace():
    """Forward and backward of two problems captured, replayed in turn with eager work between; both backwards share
    one workspace."""
    probs = [problem(51, 2, 300, 300, 8, 2, 128, "bf16"), problem(52, 1, 129, 260, 4, 4, 64, "bf16")]
    want, graphs, kept = [], [], []
    work = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    for q, k, v, dO in probs:
        want.append(run(q, k, v, dO))
        again = run(q, k, v, dO)
        assert torch.equal(want[-1][0], again[0]) and all(torch.equal(want[-1][2][n], again[2][n]) for n in again[2])
    for q, k, v, dO in probs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = g.attention_forward(q, k, v)
            gr = g.attention_backward(q, k, v, o, lse, dO, workspace=work)
        graphs.append(graph)
        kept.append((o, lse, gr))
    for i in range(4):
        for (o, lse, gr) in kept:
            for t in (o, lse, *gr.values()):
                t.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        run(*probs[i % 2])
        torch.cuda.synchronize()
        for (o, lse, gr), (wo, wl, wg) in zip(kept, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl) and all(torch.equal(gr[n], wg[n]) for n in gr), i


def test_streams_and_given_outputs():
    q, k, v, dO = problem(61, 1, 200, 200, 4, 2, 64, "bf16")
    o, lse, gr = run(q, k, v, dO)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = torch.empty_like(o), torch.empty_like(lse)
    g2 = {n: torch.empty_like(x) for n, x in gr.items()}
    g.attention_forward(q, k, v, o=o2, lse=l2, stream=side)
    r = g.attention_backward(q, k, v, o2, l2, dO, grads=g2, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and all(r[n] is g2[n] and torch.equal(gr[n], g2[n]) for n in gr)


def test_long_sequences_against_rows_of_the_plain_form():
    """16384 tokens: some rows of o and dq, and some keys' gradients from a dO that is zero but for late rows."""
    T, H, Hkv, d = 16384, 2, 1, 128
    rng = np.random.default_rng(71)
    q, k, v, dO = (rand(rng, 1, T, h, d) for h in (H, Hkv, Hkv, H))
    dO[:, :-40] = 0
    o, lse, gr = run(q, k, v, dO)
    scale, sel = float(np.float32(d ** -0.5)), slice(T - 40, T)
    ref = R.grouped(q[0, sel], k[0], v[0], dO[0, sel], scale, True, 0, q.dtype)
    R.hold("long o", o[0, sel], *ref["o"])
    R.hold("long lse", lse[0, :, sel], *ref["lse"])
    R.hold("long dq", gr["dq"][0, sel], *ref["dq"])
    R.hold("long dk", gr["dk"][0], *ref["dk"])
    R.hold("long dv", gr["dv"][0], *ref["dv"])


def test_offsets_past_32_bits():
    """A key tensor of more than 2^32 bytes with far strides; the last sequence against itself alone."""
    d, Hkv, T, far = 128, 1, 1100, 1 << 21
    base = torch.empty(T * far + d, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(81)
    q, kv = rand(rng, 1, T, 2, d), rand(rng, 1, T, Hkv, d)
    k = base[:T * far].view(1, T, 1, far)[..., :d]
    k.copy_(kv)
    o, lse, gr = run(q, k, k, torch.ones_like(q))
    o2, lse2, gr2 = run(q, kv, kv, torch.ones_like(q))
    assert k.stride(1) * T * 2 > 1 << 32
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(gr[n], gr2[n]) for n in gr)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,T,H,Hkv", [(64, 260, 2, 1), (128, 260, 2, 1), (64, 131, 72, 36)])
def test_gradients_under_large_scores(d, T, H, Hkv, dtype):
    """Scores of several hundred, so that probabilities come from differences of large numbers: the gradients too are
    held to their bounds. Sizes for which those hold (a score off by less than 0.02)."""
    q, k, v, dO = problem(d + T, 1, T, T, H, Hkv, d, dtype)
    k[0, ::61] *= 30 if d == 64 else 20
    k[0, :64] *= 4
    scale = 0.5 if d == 64 else 0.25
    Q, K = R.f64(q[0]), R.f64(k[0])
    off = max((np.abs(Q[:, h]) @ np.abs(K[:, h * Hkv // H]).T).max() for h in range(H)) * scale * (d + 8) * R.U
    assert off < 0.018 and np.abs(scale * Q[:, 0] @ K[:, 0].T).max() > 300
    o, lse, gr = run(q, k, v, dO, scale=scale)
    # Probabilities below 2^-126, the smallest normal number of fp32, are zero (they reach e^-1000 here), and so are
    # products and outputs: an error of 2^-126 in each of the T H probabilities and gradients of scores, times |dp - delta|
    # of at most twice the largest |dO| |v| sum and the largest factor of the last product, and in each output.
    size = max(float(x.abs().max()) for x in (q, k, v, dO))
    under = 2.0 ** -126 * (1 + T * H * 2 * d * size ** 3)
    ref = R.grouped(q[0], k[0], v[0], dO[0], scale, True, 0, q.dtype)
    for n, got in (("o", o[0]), ("lse", lse[0]), ("dq", gr["dq"][0]), ("dk", gr["dk"][0]), ("dv", gr["dv"][0])):
        R.hold(f"large scores d{d} {dtype} {n}", got, ref[n][0], ref[n][1] + under)
