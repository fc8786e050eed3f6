"""Queries that see one key (gdn2_attention_backward): there p = 1 and delta = dp,
so ds, and what dq and dk have of it, is zero by definition: exactly, not to a
tolerance. What is no number still reaches the results that see it."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def tensors(seed, lead_q, lead_k, H, Hkv, d, dtype):
    rng = np.random.default_rng(seed)
    mk = lambda *s: torch.tensor(rng.standard_normal(s).astype(np.float32)).to(TYPES[dtype]).to(DEV)  # noqa: E731
    return mk(*lead_q, H, d), mk(*lead_k, Hkv, d), mk(*lead_k, Hkv, d), mk(*lead_q, H, d)


def zero(*ts):
    return all(int(torch.count_nonzero(t)) == 0 for t in ts)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T,S,H,Hkv,window,causal", [
    (5, 1, 1, 4, 4, 0, True), (2, 1, 1, 8, 1, 0, False), (1, 200, 200, 4, 2, 1, True), (2, 70, 130, 6, 3, 1, True),
    (1, 130, 70, 4, 2, 1, True), (3, 97, 1, 4, 2, 0, False), (2, 97, 1, 4, 2, 0, True), (4, 131, 131, 72, 36, 1, True)])
def test_every_query_sees_one_key(B, T, S, H, Hkv, window, causal, d, dtype):
    q, k, v, dO = tensors(T + S, (B, T), (B, S), H, Hkv, d, dtype)
    o, lse = g.attention_forward(q, k, v, causal=causal, window=window)
    gr = g.attention_backward(q, k, v, o, lse, dO, causal=causal, window=window)
    torch.cuda.synchronize()
    assert zero(gr["dq"], gr["dk"]) and not zero(gr["dv"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[1], [1] * 70, [0, 1, 0, 1, 1]])
def test_packed_sequences_of_one_token(lengths, dtype):
    T = sum(lengths)
    q, k, v, dO = tensors(T, (T,), (T,), 4, 2, 64, dtype)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lengths))), dtype=torch.int32, device=DEV)
    o, lse = g.attention_forward_varlen(q, k, v, cu)
    gr = g.attention_backward_varlen(q, k, v, o, lse, dO, cu)
    torch.cuda.synchronize()
    assert zero(gr["dq"], gr["dk"]) and not zero(gr["dv"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,S,H,Hkv", [(5, 5, 4, 2), (200, 200, 4, 1), (300, 170, 4, 2), (1500, 1500, 32, 16)])
def test_the_first_keys_own_query(T, S, H, Hkv, d, dtype):
    """One query of a causal sequence sees the first key alone; with a gradient of its own result only, dq and dk are zero."""
    q, k, v, dO = tensors(T, (1, T), (1, S), H, Hkv, d, dtype)
    row = T - S
    keep = dO.clone()
    dO.zero_()
    dO[:, row] = keep[:, row]
    o, lse = g.attention_forward(q, k, v)
    gr = g.attention_backward(q, k, v, o, lse, dO)
    full = g.attention_backward(q, k, v, o, lse, keep)
    torch.cuda.synchronize()
    assert zero(gr["dq"], gr["dk"]) and not zero(gr["dv"][:, 0]) and zero(gr["dv"][:, 1:])
    assert zero(full["dq"][:, row]) and bool((full["dq"][:, row + 1:] != 0).any(-1).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5])
def test_values_that_are_no_number_stay(T, dtype):
    for which in ("q", "v", "dO"):
        t = dict(zip(("q", "k", "v", "dO"), tensors(7, (1, T), (1, T), 2, 1, 64, dtype)))
        t[which][0, 0, 0, 3] = float("nan")
        o, lse = g.attention_forward(t["q"], t["k"], t["v"])
        gr = g.attention_backward(t["q"], t["k"], t["v"], o, lse, t["dO"])
        torch.cuda.synchronize()
        assert torch.isnan(gr["dq"][0, 0, 0]).all() and torch.isnan(gr["dk"][0, 0]).all(), which
        if which != "v":  # the other query head, and the queries after it
            assert torch.isfinite(gr["dq"][0, :, 1]).all() and torch.isfinite(gr["dq"][0, 1:, 0]).all(), which
