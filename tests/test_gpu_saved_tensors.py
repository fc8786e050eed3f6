"""Gradients of views of a fused projection under hooks on saved tensors, which
return dense tensors where the forward had views: the same bits as without."""
import pytest
import torch

import gated_delta_rule_83_amd as g

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
H, HK, D = 4, 2, 64


def hooks(kind):
    if kind == "cpu":
        return torch.autograd.graph.save_on_cpu()
    return torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.clone())


def parts(x):
    return [t.unflatten(-1, (-1, D)) for t in x.split([H * D, HK * D, HK * D], -1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["clone", "cpu"])
@pytest.mark.parametrize("packed", [False, True])
def test_attention(packed, kind, dtype):
    torch.manual_seed(1)
    x = torch.randn(*((150,) if packed else (2, 150)), (H + 2 * HK) * D, device=DEV).to(TYPES[dtype])
    cu = torch.tensor([0, 40, 40, 150], dtype=torch.int32, device=DEV)
    dO = torch.randn(*x.shape[:-1], H, D, device=DEV).to(x.dtype)

    def step():
        leaf = x.clone().requires_grad_()
        q, k, v = parts(leaf)
        o = g.attention_varlen(q, k, v, cu, window=60) if packed else g.attention(q, k, v)
        return lambda: torch.autograd.grad(o, leaf, dO)[0]

    plain = step()()
    with hooks(kind):
        finish = step()
    got = finish()
    torch.cuda.synchronize()
    assert torch.equal(got, plain)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["clone", "cpu"])
def test_rotary(kind, dtype):
    torch.manual_seed(2)
    x, w = torch.randn(2, 150, (H + 2 * HK) * D, device=DEV).to(TYPES[dtype]), torch.randn(D, device=DEV)
    pos = torch.arange(300, dtype=torch.int32, device=DEV).view(2, 150)
    f = 1e4 ** (-torch.arange(0, D, 2, device=DEV) / D)
    gq, gk = (torch.randn(2, 150, h, D, device=DEV).to(x.dtype) for h in (H, HK))

    def step():
        leaf, weight = x.clone().requires_grad_(), w.clone().requires_grad_()
        q, k, _ = parts(leaf)
        out = g.rotary(q, k, pos, f, weight, weight)
        return lambda: torch.autograd.grad(out, (leaf, weight), (gq, gk))

    plain = step()()
    with hooks(kind):
        finish = step()
    got = finish()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, plain))


def test_a_layout_that_no_call_takes_is_refused():
    """A hook that returns a batch's tokens not one distance apart."""
    x = torch.randn(2, 30, (H + 2 * HK) * D, device=DEV, requires_grad=True)
    pos, f = torch.arange(60, dtype=torch.int32, device=DEV).view(2, 30), torch.ones(D // 2, device=DEV)

    def unpack(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1) if t.dim() == 4 else t

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        q, k, v = parts(x)
        outs = g.attention(q, k, v), g.rotary(q, k, pos, f)[0]
    for y in outs:
        with pytest.raises(ValueError, match="one distance apart|contiguous"):
            torch.autograd.grad(y.sum(), x, retain_graph=True)
