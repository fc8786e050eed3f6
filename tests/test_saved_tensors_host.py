"""Autograd functions whose inputs may be views of a fused projection, under hooks
on saved tensors (activations kept elsewhere until the backward): what comes back
is dense, so the backward has to be told the distances of the tokens that it
gets, not those of the forward's. On the CPU, with the library's calls recorded."""
import pytest
import torch

import gated_delta_rule_83_amd as g

H, HK, D = 4, 2, 64


@pytest.fixture
def recorded(monkeypatch):
    """Calls of the library in place of launches: (name, desc, pointers)."""
    calls = []

    class here:
        def __init__(self, *a):
            pass

        def __enter__(self):
            return 0

        def __exit__(self, *a):
            return False

    def record(name):
        def call(desc, *ptrs):
            calls.append((name, desc, ptrs))
            return g.GDN2_OK
        return call

    monkeypatch.setattr(g, "_check", lambda t, name, dtype=None: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    for mod in (g.attention_ops, g.rotary_ops):
        monkeypatch.setattr(mod, "launch_on", here)
        monkeypatch.setattr(mod, "want_tokens", lambda t, *a: t.stride(-3))
        for nm in g.EXPORTED:
            if hasattr(mod, nm) and not nm.endswith("_bytes"):
                monkeypatch.setattr(mod, nm, record(nm))
    return calls


def parts(lead):
    leaf = torch.randn(*lead, (H + 2 * HK) * D, requires_grad=True)
    return leaf, [x.unflatten(-1, (-1, D)) for x in leaf.split([H * D, HK * D, HK * D], -1)]


@pytest.mark.parametrize("hooked", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_attention(recorded, packed, hooked):
    leaf, (q, k, v) = parts((10,) if packed else (2, 5))
    seen = {}

    def unpack(t):
        t = t.clone() if hooked else t
        seen[t.data_ptr()] = t
        return t

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        o = g.attention_varlen(q, k, v, torch.tensor([0, 4, 10], dtype=torch.int32)) if packed else g.attention(q, k, v)
    o.sum().backward()
    (_, fwd, _), (name, bwd, ptrs) = recorded
    assert "backward" in name and (fwd.stride_q, fwd.stride_k, fwd.stride_v) == ((H + 2 * HK) * D,) * 3
    for p, stride, heads in zip(ptrs[2 * packed:], (bwd.stride_q, bwd.stride_k, bwd.stride_v), (H, HK, HK)):
        assert seen[p].shape[-2] == heads and stride == seen[p].stride(-3)
    assert leaf.grad.shape == leaf.shape


@pytest.mark.parametrize("hooked", [False, True])
def test_rotary(recorded, hooked):
    leaf, (q, k, _) = parts((2, 5))
    seen = {}

    def unpack(t):
        t = t.clone() if hooked else t
        seen[t.data_ptr()] = t
        return t

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        a, b = g.rotary(q, k, torch.zeros(2, 5, dtype=torch.int32), torch.ones(D // 2))
    (a.sum() + b.sum()).backward()
    (_, fwd, _), (name, bwd, ptrs) = recorded
    assert "backward" in name and (fwd.stride_q, fwd.stride_k) == ((H + 2 * HK) * D,) * 2
    for p, stride, heads in zip(ptrs, (bwd.stride_q, bwd.stride_k), (H, HK)):
        assert seen[p].shape[-2] == heads and stride == seen[p].stride(-3)
