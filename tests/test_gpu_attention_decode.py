"""One token over a paged key-value cache (gdn2_attention_decode) and the cache's
writes (gdn2_kv_cache_store), against the 64-bit plain form over each sequence's
tokens; bounds from attention_ref (a span's and a wave's partial sums are joined
in fp32: no more roundings than a row of one pass has)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def problem(seed, lengths, H, Hkv, d, page, dtype, room=0):
    """A cache filled with NaN but for the sequences' tokens, its pages dealt out in random order."""
    rng = np.random.default_rng(seed)
    dt = R.TYPES[dtype]
    need = [-(-n // page) for n in lengths]
    M, P = max(max(need), 1) + room, sum(need) + 3
    order = rng.permutation(P)
    table = np.full((len(lengths), M), -1, np.int32)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
    kc, vc = (torch.full((P, Hkv, page, d), float("nan"), dtype=dt, device=DEV) for _ in range(2))
    toks = []
    for n, length in enumerate(lengths):
        k, v = (torch.tensor(rng.standard_normal((length, Hkv, d)).astype(np.float32)).to(dt).to(DEV) for _ in range(2))
        t = np.arange(length)
        pg, row = torch.tensor(table[n, t // page], device=DEV).long(), torch.tensor(t % page, device=DEV)
        kc[pg, :, row], vc[pg, :, row] = k, v
        toks.append((k, v))
    q = torch.tensor(rng.standard_normal((len(lengths), 1, H, d)).astype(np.float32)).to(dt).to(DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return q, kc, vc, ints(table), ints(lengths), toks


def check(name, o, q, toks, window=0, scale=None):
    scale = float(np.float32(q.shape[-1] ** -0.5 if scale is None else scale))
    for n, (k, v) in enumerate(toks):
        ref = R.grouped(q[n], k, v, None, scale, True, window, q.dtype)
        R.hold(f"{name} {n}", o[n], *ref["o"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 8, 16, 32, 64, 256])
@pytest.mark.parametrize("lengths", [[1], [0, 5, 0], [31, 32, 33], [63, 64, 65, 127, 128, 129], [300, 1, 1000, 17]])
def test_decode(lengths, page, d, dtype):
    q, kc, vc, pages, ln, toks = problem(sum(lengths) + page, lengths, 4, 2, d, page, dtype)
    o = g.attention_decode(q, kc, vc, pages, ln)
    torch.cuda.synchronize()
    check(f"decode page {page} d{d} {dtype}", o, q, toks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (40, 2), (32, 4)])
def test_head_layouts(H, Hkv, dtype):
    q, kc, vc, pages, ln, toks = problem(H, [200, 37], H, Hkv, 64, 16, dtype)
    o = g.attention_decode(q, kc, vc, pages, ln)
    torch.cuda.synchronize()
    check(f"decode heads {H}/{Hkv}", o, q, toks)


@pytest.mark.parametrize("page", [4, 64])
@pytest.mark.parametrize("window", [1, 31, 32, 33, 100, 129, 5000])
def test_window(window, page):
    q, kc, vc, pages, ln, toks = problem(window, [700, 100, 1, 32, 0], 8, 2, 128, page, "bf16")
    o = g.attention_decode(q, kc, vc, pages, ln, window=window)
    torch.cuda.synchronize()
    check(f"decode window {window}", o, q, toks, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_caches_split_and_joined(dtype):
    """Spans of several lengths, empty ones among them, and a table with room for far more than there is."""
    q, kc, vc, pages, ln, toks = problem(5, [20000, 130, 0, 4097], 4, 2, 128, 64, dtype, room=500)
    o = g.attention_decode(q, kc, vc, pages, ln)
    again = g.attention_decode(q, kc, vc, pages, ln, workspace=torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(o, again)  # the workspace's contents are nothing to it
    check(f"decode long {dtype}", o, q, toks)


def test_bad_pages_and_lengths():
    """Pages outside the cache are not seen; lengths are clamped to the table."""
    q, kc, vc, pages, ln, toks = problem(7, [200, 90, 64], 4, 2, 64, 32, "bf16")
    pages[0, 2], pages[0, 4] = -5, 10 ** 9
    pages[1] = -1
    keep = torch.tensor([t for t in range(200) if t // 32 not in (2, 4)], device=DEV)
    ln2 = torch.tensor([200, 90, 10 ** 6], dtype=torch.int32, device=DEV)
    o = g.attention_decode(q, kc, vc, pages, ln2)
    zero = g.attention_decode(q, kc, vc, pages, torch.tensor([-7, 0, -2 ** 31], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert (zero == 0).all() and (o[1] == 0).all()
    # sequence 2's other pages are -1: its 64 tokens are what is seen
    check("decode bad pages", o[[0, 2]], q[[0, 2]], [tuple(x[keep] for x in toks[0]), toks[2]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length", [1, 33, 100, 129, 3000])
def test_scores_that_are_no_number(length, dtype):
    """A query that is no number, and a last key that is alone in its wave: no result hides them."""
    q, kc, vc, pages, ln, _ = problem(10, [length, length], 4, 2, 64, 32, dtype)
    q[0, 0, 1, 7] = float("nan")
    t = length - 1
    kc[pages[1, t // 32].long(), 0, t % 32, 3] = float("nan")
    o = g.attention_decode(q, kc, vc, pages, ln)
    torch.cuda.synchronize()
    assert torch.isnan(o[0, 0, 1]).all() and torch.isfinite(o[0, 0, [0, 2, 3]]).all()
    assert torch.isnan(o[1, 0, :2]).all() and torch.isfinite(o[1, 0, 2:]).all()


@pytest.mark.parametrize("page", [8, 64])
def test_values_that_are_no_number(page):
    q, kc, vc, pages, ln, toks = problem(9, [100, 100], 4, 2, 64, page, "bf16")
    t = 40
    vc[pages[0, t // page].long(), 1, t % page, 3] = float("nan")
    kc[pages[1, t // page].long(), 0, t % page, 3] = float("nan")
    o = g.attention_decode(q, kc, vc, pages, ln)
    w = g.attention_decode(q, kc, vc, pages, ln, window=59)
    torch.cuda.synchronize()
    assert torch.isnan(o[0, 0, 2:, 3]).all() and torch.isfinite(o[0, 0, :2]).all() and torch.isfinite(o[0, 0, 2:, 4:]).all()
    assert torch.isnan(o[1, 0, :2]).all() and torch.isfinite(o[1, 0, 2:]).all()
    assert torch.isfinite(w).all()  # behind the window


def test_offsets_past_32_bits():
    P, Hkv, page, d = 140000, 2, 64, 128
    kc = torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    q, k0, v0, pages, ln, toks = problem(11, [150], 4, Hkv, d, page, "bf16")
    far = torch.tensor([[P - 1, 3, P - 2]], dtype=torch.int32, device=DEV)
    for i in range(3):
        kc[far[0, i].long()], vc[far[0, i].long()] = k0[pages[0, i].long()], v0[pages[0, i].long()]
    o = g.attention_decode(q, kc, vc, far, ln)
    want = g.attention_decode(q, k0, v0, pages, ln)
    torch.cuda.synchronize()
    assert kc.numel() * 2 > 1 << 32 and torch.equal(o, want)
    # and a write there
    k, v = (torch.randn(1, 1, Hkv, d, device=DEV).to(torch.bfloat16) for _ in range(2))
    g.kv_cache_store(k, v, far, ln, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc[P - 2, :, 149 % 64], k[0, 0]) and torch.equal(vc[P - 2, :, 149 % 64], v[0, 0])


def test_a_replayed_graph_takes_new_lengths():
    q, kc, vc, pages, ln, toks = problem(13, [500, 900], 8, 2, 128, 64, "bf16")
    o = g.attention_decode(q, kc, vc, pages, ln)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = g.attention_decode(q, kc, vc, pages, ln)
    for i in range(4):
        short = torch.tensor([500 - 100 * i, 900 - 300 * i], dtype=torch.int32, device=DEV)
        ln.copy_(short)
        got.fill_(float("nan"))
        graph.replay()
        want = g.attention_decode(q, kc, vc, pages, short)
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
    del o


# ------------------------------------------------------------------ the cache's writes
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("d,Hkv", [(64, 1), (64, 3), (128, 2)])
def test_store_packed_prompts(d, Hkv, page, dtype):
    """Prompts behind prefixes; every other row of the cache as it was, tokens of no sequence nowhere."""
    dt, rng = R.TYPES[dtype], np.random.default_rng(page + d)
    counts, past = [5, 0, 70, 1, 33], [0, 9, 130, 64, 31]
    lengths = [a + b for a, b in zip(counts, past)]
    need = [-(-n // page) for n in lengths]
    P = sum(need) + 4
    order = rng.permutation(P).astype(np.int32)
    table = np.full((5, max(need)), -1, np.int32)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
    cu = np.concatenate(([0], np.cumsum(counts))).astype(np.int32) + 2
    T = int(cu[-1]) + 3
    mk = lambda *s: torch.tensor(rng.standard_normal(s).astype(np.float32)).to(dt).to(DEV)  # noqa: E731
    fused = mk(T, 2 * Hkv * d)
    k, v = (x.unflatten(-1, (Hkv, d)) for x in fused.split([Hkv * d, Hkv * d], -1))
    kc, vc = mk(P, Hkv, page, d), mk(P, Hkv, page, d)
    wk, wv = kc.clone(), vc.clone()
    for n in range(5):
        for i in range(counts[n]):
            t = past[n] + i
            wk[int(table[n, t // page]), :, t % page] = k[int(cu[n]) + i]
            wv[int(table[n, t // page]), :, t % page] = v[int(cu[n]) + i]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    g.kv_cache_store(k, v, ints(table), ints(lengths), kc, vc, cu_seqlens=ints(cu))
    torch.cuda.synchronize()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_store_one_token_each_and_places_that_are_none():
    kc, vc = g.kv_cache_empty(6, 2, 64, page=16)
    k, v = (torch.randn(7, 1, 2, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    pages = torch.tensor([[0, 1], [2, 3], [-1, 4], [9, 4], [5, -1], [5, -1], [5, -1]], dtype=torch.int32, device=DEV)
    #                      row 15   page 3   none     none     length 0  past the table, negative
    lengths = torch.tensor([16, 17, 3, 8, 0, 33, -4], dtype=torch.int32, device=DEV)
    g.kv_cache_store(k, v, pages, lengths, kc, vc)
    torch.cuda.synchronize()
    wk, wv = torch.zeros_like(kc), torch.zeros_like(vc)
    wk[0, :, 15], wk[3, :, 0], wv[0, :, 15], wv[3, :, 0] = k[0, 0], k[1, 0], v[0, 0], v[1, 0]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,length", [(5, 1, 640), (1, 1, 600), (3, 3, 897)])
def test_an_odd_number_of_heads_and_spans(H, Hkv, length, d, dtype):
    """The spans' outputs lie behind an odd number of statistics."""
    q, kc, vc, pages, ln, toks = problem(H + length, [length], H, Hkv, d, 32, dtype)
    o = g.attention_decode(q, kc, vc, pages, ln)
    torch.cuda.synchronize()
    check(f"decode odd {H} {length}", o, q, toks)


@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("H,Hkv,d,length", [(16, 2, 128, 3000), (4, 4, 64, 400), (8, 1, 64, 70)])
def test_probabilities_keep_more_than_the_outputs_type(H, Hkv, d, length, page):
    """bf16: a probability is held as an operand in two parts of 8 bits, off by 2^-15 of itself at most (the second part's
    rounding, 2^-8 of 2^-7), so a result is off by its own rounding, 2^-8, and next to nothing else."""
    q, kc, vc, pages, ln, toks = problem(H + length, [length, length // 2], H, Hkv, d, page, "bf16")
    o = g.attention_decode(q, kc, vc, pages, ln)
    torch.cuda.synchronize()
    scale, U, h = float(np.float32(d ** -0.5)), R.U, 2.0 ** -8
    for n, (k, v) in enumerate(toks):
        Q, K, V = R.f64(q[n, 0]), R.f64(k), R.f64(v)
        for head in range(H):
            a, b = K[:, head * Hkv // H], V[:, head * Hkv // H]
            s = scale * a @ Q[head]
            off = scale * (d + 8) * U * (np.abs(a) @ np.abs(Q[head])) + 6 * U * np.abs(s)
            p = np.exp(s - s.max())
            p /= p.sum()
            rel = 2.1 * off + 8 * U
            rel = rel + (p * rel).sum() + (len(s) / 16 + 16) * U + 2.0 ** -15
            tol = (p * rel) @ np.abs(b) + (len(s) + 16) * U * (p @ np.abs(b))
            ref = p @ b
            R.hold(f"decode in two parts {n} {head}", o[n, 0, head], ref, tol + (h + 2 * U) * (np.abs(ref) + tol))
