"""Infinite scores and values in places that a query sees (gdn2_attention_*,
gdn2_attention_decode), at the edge of what it sees and inside. Bounds from
attention_ref."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


def problem(seed, B, T, H, Hkv, d, dtype):
    rng = np.random.default_rng(seed)
    mk = lambda h: torch.tensor(rng.standard_normal((B, T, h, d)).astype(np.float32)).to(R.TYPES[dtype]).to(DEV)  # noqa: E731
    return mk(H), mk(Hkv), mk(Hkv), mk(H)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T,H,Hkv,first", [(1, 40, 4, 2, 10), (1, 300, 4, 2, 150), (2, 131, 72, 36, 70)])
def test_scores_of_minus_infinity_alone(B, T, H, Hkv, first, d, dtype):
    """Products with the first keys overflow: queries that see those alone are as queries without keys, and the others
    as if those keys were not there."""
    q, k, v, dO = problem(T + d, B, T, H, Hkv, d, dtype)
    q[..., 0], k[:, :first, :, 0], k[:, first:, :, 0] = 1e30, -1e30, 0
    o, lse = g.attention_forward(q, k, v)
    gr = g.attention_backward(q, k, v, o, lse, dO)
    torch.cuda.synchronize()
    assert (o[:, :first] == 0).all() and (lse[:, :, :first] == -INF).all()
    for nm in ("dq", "dk", "dv"):
        assert (gr[nm][:, :first] == 0).all(), nm
    scale = float(np.float32(d ** -0.5))
    for b in range(B):
        ref = R.grouped(*(t[b, first:] for t in (q, k, v, dO)), scale, True, 0, q.dtype)
        for nm, got in (("o", o), ("dq", gr["dq"]), ("dk", gr["dk"]), ("dv", gr["dv"])):
            R.hold(f"after -inf {nm}", got[b, first:], *ref[nm])
        R.hold("after -inf lse", lse[b, :, first:], *ref["lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_keys(dtype):
    """The same by keys of -inf: decode over the same tokens says the same as the whole sequence's forward."""
    T, first = 90, 70
    q, k, v, _ = problem(3, 1, T, 4, 2, 64, dtype)
    q[..., 5] = q[..., 5].abs() + 1
    k[:, :first, :, 5] = -INF
    o, lse = g.attention_forward(q, k, v)
    kc, vc = g.kv_cache_empty(3, 2, 64, page=32, dtype=q.dtype, device=DEV)
    pages = torch.arange(3, dtype=torch.int32, device=DEV)[None]
    whole = torch.tensor([T], dtype=torch.int32, device=DEV)
    g.kv_cache_store(k[0], v[0], pages, whole, kc, vc, cu_seqlens=torch.tensor([0, T], dtype=torch.int32, device=DEV))
    for n in (1, 33, first, first + 1, T):
        one = g.attention_decode(q[:, n - 1:n], kc, vc, pages, torch.full_like(whole, n))
        torch.cuda.synchronize()
        if n <= first:
            assert (one == 0).all() and (o[:, n - 1] == 0).all() and (lse[:, :, n - 1] == -INF).all()
        else:
            assert torch.isfinite(one).all() and torch.isfinite(lse[:, :, n - 1]).all()
            ref = R.grouped(q[0, n - 1:n], k[0, first:n], v[0, first:n], None, float(np.float32(0.125)), True, 0, q.dtype)["o"]
            R.hold(f"decode {n}", one[0], *ref)
            R.hold(f"forward {n}", o[0, n - 1:n], *ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("B,T,H,Hkv,place,window", [(1, 400, 2, 1, 70, 0), (1, 400, 2, 1, 64, 0), (1, 400, 2, 1, 40, 90),
                                                     (2, 300, 72, 36, 100, 0), (2, 300, 72, 36, 1, 70)])
def test_an_infinite_value(B, T, H, Hkv, place, window, sign, d, dtype):
    """Whichever tile it lies in, wholly seen or at an edge: the queries that see it have that infinity."""
    q, k, v, dO = problem(T + place, B, T, H, Hkv, d, dtype)
    o, lse = g.attention_forward(q, k, v, window=window)
    v[:, place, :, 7] = sign * INF
    o2, lse2 = g.attention_forward(q, k, v, window=window)
    torch.cuda.synchronize()
    end = min(T, place + window) if window else T
    assert torch.equal(lse, lse2) and (o2[:, place:end, :, 7] == sign * INF).all()
    o[:, place:end, :, 7] = o2[:, place:end, :, 7]
    assert torch.equal(o, o2)
    # beside the opposite one: NaN for who sees both
    v[:, place + 20, :, 7] = -sign * INF
    o3, _ = g.attention_forward(q, k, v, window=window)
    torch.cuda.synchronize()
    assert torch.isnan(o3[:, place + 20:end, :, 7]).all() and (o3[:, place:place + 20, :, 7] == sign * INF).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("B,T,H,Hkv,place,window", [(1, 400, 2, 1, 330, 0), (1, 400, 2, 1, 200, 70), (2, 300, 72, 36, 250, 0)])
def test_an_infinite_gradient(B, T, H, Hkv, place, window, sign, d, dtype):
    """dv of every key that its query sees has that infinity, its dq and their dk are NaN; all else is as it was."""
    q, k, v, dO = problem(T + place, B, T, H, Hkv, d, dtype)
    o, lse = g.attention_forward(q, k, v, window=window)
    gr = g.attention_backward(q, k, v, o, lse, dO, window=window)
    dO[:, place, 0, 7] = sign * INF
    g2 = g.attention_backward(q, k, v, o, lse, dO, window=window)
    torch.cuda.synchronize()
    first = max(0, place - window + 1) if window else 0
    assert (g2["dv"][:, first:place + 1, 0, 7] == sign * INF).all()
    assert torch.isnan(g2["dq"][:, place, 0]).all() and torch.isnan(g2["dk"][:, first:place + 1, 0]).all()
    gr["dv"][:, first:place + 1, 0, 7] = sign * INF
    for t in (gr, g2):
        t["dq"][:, place, 0], t["dk"][:, first:place + 1, 0] = 0, 0
    # (the tiles beside it are computed again, in the same order)
    assert all(torch.equal(gr[n], g2[n]) for n in gr)


@pytest.mark.parametrize("page", [8, 64])
def test_an_infinite_value_decoded(page):
    q, k, v, _ = problem(5, 1, 200, 4, 2, 64, "bf16")
    v[0, 90, 1, 3] = -INF
    kc, vc = g.kv_cache_empty(200 // page + 1, 2, 64, page=page, device=DEV)
    pages = torch.arange(200 // page + 1, dtype=torch.int32, device=DEV)[None]
    ln = torch.tensor([200], dtype=torch.int32, device=DEV)
    g.kv_cache_store(k[0], v[0], pages, ln, kc, vc, cu_seqlens=torch.tensor([0, 200], dtype=torch.int32, device=DEV))
    o = g.attention_decode(q[:, 199:], kc, vc, pages, ln)
    w = g.attention_decode(q[:, 199:], kc, vc, pages, ln, window=109)
    torch.cuda.synchronize()
    assert (o[0, 0, 2:, 3] == -INF).all() and torch.isfinite(o[0, 0, :2]).all() and torch.isfinite(o[0, 0, :, 4:]).all()
    assert torch.isfinite(w).all()
