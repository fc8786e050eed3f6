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
