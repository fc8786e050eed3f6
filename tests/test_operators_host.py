"""Host checks of the linear recurrence, the norms and the state cache: every
refused call returns its status before any HIP call (made-up addresses that
are never read), and the torch conveniences refuse what would be read or
written out of its bounds before the library is reached."""
import ctypes

import pytest
import torch

import gated_delta_rule_83_amd as g

FAKE, EACH = 1 << 40, 1 << 32  # distinct made-up buffers, EACH bytes apart


def fakes(n):
    return [FAKE + i * EACH for i in range(n)]


# ------------------------------------------------------------------ C ABI: linear recurrence
def lin(B=2, T=300, D=64, gates=0, dtype=1):
    return g.gdn2_linear_desc(B, T, D, gates, dtype)


def fwd(d, p=None, ws=True):
    # x, a, b, h0, o, h_T, ck
    return g.gdn2_linear_forward(d, *(p or fakes(7)), FAKE - EACH if ws else 0, 1 << 30 if ws else 0, 0)


def fwd_varlen(d, p=None):
    return g.gdn2_linear_forward_varlen(d, *(p or fakes(8)), FAKE - EACH, 1 << 30, 0)


def bwd(d, p=None, ws=1 << 30):
    # x, a, b, h0, ck, dO, dh_T, dx, da, db, dh0
    return g.gdn2_linear_backward(d, *(p or fakes(11)), FAKE - EACH if ws else 0, ws, 0)


def put(p, **at):
    p = list(p)
    for k, v in at.items():
        p[int(k[1:])] = v
    return p


BAD_LINEAR = [(None, g.GDN2_ERR_NULL_POINTER), (lin(dtype=2), g.GDN2_ERR_BAD_DTYPE), (lin(B=-1), g.GDN2_ERR_BAD_SHAPE),
              (lin(T=-1), g.GDN2_ERR_BAD_SHAPE), (lin(D=0), g.GDN2_ERR_BAD_SHAPE), (lin(gates=4), g.GDN2_ERR_UNSUPPORTED),
              (lin(gates=-1), g.GDN2_ERR_UNSUPPORTED), (lin(T=2 ** 31 - 1), g.GDN2_ERR_UNSUPPORTED),
              (lin(B=2 ** 31 - 1, D=2 ** 31 - 1), g.GDN2_ERR_UNSUPPORTED), (lin(D=2 ** 22 + 1), g.GDN2_ERR_UNSUPPORTED), (lin(B=2 ** 24), g.GDN2_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("desc,status", BAD_LINEAR)
def test_linear_descriptions(desc, status):
    assert fwd(desc) == status and fwd_varlen(desc) == status and bwd(desc) == status
    assert g.gdn2_linear_step(desc, *fakes(6)) == status
    for query in (g.gdn2_linear_forward_workspace_bytes, g.gdn2_linear_forward_varlen_workspace_bytes,
                  g.gdn2_linear_backward_workspace_bytes, g.gdn2_linear_backward_varlen_workspace_bytes):
        assert query(desc) == 0


def test_linear_pointers():
    f = fakes(7)
    for i in (0, 1, 2):
        assert fwd(lin(), put(f, **{f"_{i}": 0})) == g.GDN2_ERR_NULL_POINTER, i
    assert fwd(lin(), f[:4] + [0, 0, 0]) == g.GDN2_ERR_NULL_POINTER  # nothing to compute
    for i, off in ((0, 1), (1, 2), (2, 2), (3, 2), (4, 1), (5, 2), (6, 2)):  # less than an element off
        assert fwd(lin(), put(f, **{f"_{i}": f[i] + off})) == g.GDN2_ERR_BAD_SHAPE, i
    for out in (4, 6):
        for i in (0, 1, 2, 3):
            assert fwd(lin(), put(f, **{f"_{out}": f[i] + 64})) == g.GDN2_ERR_ALIAS, (out, i)
    assert fwd(lin(), put(f, _5=f[3] + 64)) == g.GDN2_ERR_ALIAS  # h_T partly h0
    assert fwd(lin(), put(f, _5=f[4])) == g.GDN2_ERR_ALIAS      # h_T in o
    f = fakes(8)
    assert fwd_varlen(lin(), put(f, _0=0)) == g.GDN2_ERR_NULL_POINTER
    assert fwd_varlen(lin(), put(f, _0=f[0] + 2)) == g.GDN2_ERR_BAD_SHAPE
    assert fwd_varlen(lin(), put(f, _5=f[0])) == g.GDN2_ERR_ALIAS  # o over the offsets
    s = fakes(6)  # x, a, b, h, h_out, o
    for i in (0, 1, 2, 3, 4, 5):
        assert g.gdn2_linear_step(lin(T=1), *put(s, **{f"_{i}": 0})) == g.GDN2_ERR_NULL_POINTER, i
    assert g.gdn2_linear_step(lin(T=2), *s) == g.GDN2_ERR_BAD_SHAPE
    assert g.gdn2_linear_step(lin(T=1), *put(s, _4=s[3] + 4)) == g.GDN2_ERR_ALIAS
    assert g.gdn2_linear_step(lin(T=1), *put(s, _5=s[3])) == g.GDN2_ERR_ALIAS
    assert g.gdn2_linear_step(lin(T=1), *put(s, _5=s[0])) == g.GDN2_ERR_ALIAS


def test_linear_backward_pointers_and_workspace():
    f = fakes(11)
    for i in (0, 1, 2, 5, 7, 8, 9):
        assert bwd(lin(), put(f, **{f"_{i}": 0})) == g.GDN2_ERR_NULL_POINTER, i
    for out in (7, 8, 9, 10):
        for i in (0, 1, 2, 3, 4, 5):
            assert bwd(lin(), put(f, **{f"_{out}": f[i] + 64})) == g.GDN2_ERR_ALIAS, (out, i)
    assert bwd(lin(), put(f, _10=f[6] + 64)) == g.GDN2_ERR_ALIAS
    assert bwd(lin(), put(f, _7=f[8])) == g.GDN2_ERR_ALIAS
    need = g.gdn2_linear_backward_workspace_bytes(lin())
    assert need >= 2 * 3 * 64 * 4  # the states every 64 tokens
    assert bwd(lin(), f, need - 1) == g.GDN2_ERR_WORKSPACE and bwd(lin(), f, 0) == g.GDN2_ERR_WORKSPACE
    assert g.gdn2_linear_backward(lin(), *f, f[0], need, 0) == g.GDN2_ERR_ALIAS
    assert g.gdn2_linear_backward(lin(), *f, FAKE - EACH + 4, need, 0) == g.GDN2_ERR_BAD_SHAPE


def test_empty_batches_return_before_any_pointer_check():
    assert fwd(lin(B=0), [0] * 7, ws=False) == g.GDN2_OK
    assert fwd_varlen(lin(B=0), [0] * 8) == g.GDN2_OK
    assert bwd(lin(B=0), [0] * 11, 0) == g.GDN2_OK
    assert g.gdn2_linear_backward_varlen(lin(B=0, T=0), *[0] * 12) == g.GDN2_OK
    assert g.gdn2_linear_backward_varlen(lin(B=0), *[0] * 12) == g.GDN2_ERR_NULL_POINTER  # zeros to write
    assert g.gdn2_linear_step(lin(B=0, T=1), *[0] * 6) == g.GDN2_OK
    assert g.gdn2_norm_forward(nrm(rows=0), 0, 0, 0, 0, 0) == g.GDN2_OK
    assert g.gdn2_state_cache_store(cch(N=0), 0, 0, 0, 0) == g.GDN2_OK
    assert g.gdn2_state_cache_load(cch(N=0), 0, 0, 0, 0) == g.GDN2_OK


# ------------------------------------------------------------------ C ABI: norms
def nrm(rows=100, D=128, kind=0, dtype=1, wdtype=0, eps=1e-5):
    return g.gdn2_norm_desc(rows, D, kind, dtype, wdtype, eps)


BAD_NORM = [(None, g.GDN2_ERR_NULL_POINTER), (nrm(dtype=2), g.GDN2_ERR_BAD_DTYPE), (nrm(wdtype=-1), g.GDN2_ERR_BAD_DTYPE),
            (nrm(rows=-1), g.GDN2_ERR_BAD_SHAPE), (nrm(D=0), g.GDN2_ERR_BAD_SHAPE), (nrm(eps=-1.0), g.GDN2_ERR_BAD_SHAPE),
            (nrm(eps=float("nan")), g.GDN2_ERR_BAD_SHAPE), (nrm(eps=float("inf")), g.GDN2_ERR_BAD_SHAPE),
            (nrm(kind=2), g.GDN2_ERR_UNSUPPORTED), (nrm(rows=2 ** 62), g.GDN2_ERR_UNSUPPORTED),
            (nrm(D=2 ** 25 + 1), g.GDN2_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("desc,status", BAD_NORM)
def test_norm_descriptions(desc, status):
    assert g.gdn2_norm_forward(desc, *fakes(5)) == status
    assert g.gdn2_norm_backward(desc, *fakes(9), FAKE - EACH, 1 << 30) == status
    assert g.gdn2_norm_backward_workspace_bytes(desc) == 0


def test_norm_pointers_and_workspace():
    f = fakes(5)  # x, weight, bias, gate, y
    assert g.gdn2_norm_forward(nrm(), *put(f, _0=0)) == g.GDN2_ERR_NULL_POINTER
    assert g.gdn2_norm_forward(nrm(), *put(f, _4=0)) == g.GDN2_ERR_NULL_POINTER
    for i, off in ((0, 1), (1, 2), (2, 2), (3, 1), (4, 1)):
        assert g.gdn2_norm_forward(nrm(), *put(f, **{f"_{i}": f[i] + off})) == g.GDN2_ERR_BAD_SHAPE, i
    for i in range(4):
        assert g.gdn2_norm_forward(nrm(), *put(f, _4=f[i])) == g.GDN2_ERR_ALIAS, i
    f = fakes(9)  # x, weight, bias, gate, dy, dx, dweight, dbias, dgate
    bw = lambda p, ws=1 << 30, at=FAKE - EACH: g.gdn2_norm_backward(nrm(), *p, at, ws)
    for i in (0, 4, 5):
        assert bw(put(f, **{f"_{i}": 0})) == g.GDN2_ERR_NULL_POINTER, i
    for i in (1, 2, 3):  # a gradient of what is not there
        assert bw(put(f, **{f"_{i}": 0})) == g.GDN2_ERR_NULL_POINTER, i
    for out in (5, 6, 7, 8):
        for i in range(5):
            assert bw(put(f, **{f"_{out}": f[i]})) == g.GDN2_ERR_ALIAS, (out, i)
    need = g.gdn2_norm_backward_workspace_bytes(nrm())
    assert need > 0 and bw(f, need - 1) == g.GDN2_ERR_WORKSPACE
    assert bw(f, need, f[5]) == g.GDN2_ERR_ALIAS and bw(f, need, FAKE - EACH + 8) == g.GDN2_ERR_BAD_SHAPE


# ------------------------------------------------------------------ C ABI: state cache
def cch(N=3, P=9, rows=2048, d_v=128, fmt=0):
    return g.gdn2_cache_desc(N, P, rows, d_v, fmt)


@pytest.mark.parametrize("desc,status", [
    (None, g.GDN2_ERR_NULL_POINTER), (cch(N=-1), g.GDN2_ERR_BAD_SHAPE), (cch(P=-1), g.GDN2_ERR_BAD_SHAPE),
    (cch(rows=0), g.GDN2_ERR_BAD_SHAPE), (cch(d_v=0), g.GDN2_ERR_BAD_SHAPE), (cch(d_v=48), g.GDN2_ERR_UNSUPPORTED),
    (cch(fmt=2), g.GDN2_ERR_UNSUPPORTED), (cch(rows=2 ** 31 - 1), g.GDN2_ERR_UNSUPPORTED),
    (cch(N=2 ** 24), g.GDN2_ERR_UNSUPPORTED),
    (cch(N=2 ** 18, rows=32 * 64), g.GDN2_ERR_UNSUPPORTED)])
def test_cache_descriptions(desc, status):
    assert g.gdn2_state_cache_store(desc, *fakes(4)) == status
    assert g.gdn2_state_cache_load(desc, *fakes(4)) == status


def test_cache_pointers():
    f = fakes(4)  # store: S, slots, cache, scales
    for i in range(4):
        assert g.gdn2_state_cache_store(cch(), *put(f, **{f"_{i}": 0})) == g.GDN2_ERR_NULL_POINTER, i
        assert g.gdn2_state_cache_load(cch(), *put(f, **{f"_{i}": 0})) == g.GDN2_ERR_NULL_POINTER, i
        for j in range(4):
            if j != i:
                assert g.gdn2_state_cache_store(cch(), *put(f, **{f"_{i}": f[j]})) == g.GDN2_ERR_ALIAS, (i, j)
    for i, off in ((0, 4), (1, 2), (2, 8)):
        assert g.gdn2_state_cache_store(cch(), *put(f, **{f"_{i}": f[i] + off})) == g.GDN2_ERR_BAD_SHAPE, i


# ------------------------------------------------------------------ torch conveniences
@pytest.fixture
def host_tensors(monkeypatch):
    """CPU tensors pass the "on a GPU" check; the library refuses to be called."""
    def check(t, name, dtype=None):
        if t is None:
            return
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")

    monkeypatch.setattr(g, "_check", check)

    class here:
        def __init__(self, *a):
            pass

        def __enter__(self):
            return 0

        def __exit__(self, *a):
            return False

    def refuse(*a, **k):
        raise AssertionError("a mis-shaped call reached the library")

    for mod in (g.linear, g.norms, g.state_cache):
        monkeypatch.setattr(mod, "launch_on", here)
        for nm in g.EXPORTED:
            if hasattr(mod, nm) and not nm.endswith("_bytes"):
                monkeypatch.setattr(mod, nm, refuse)


f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


def z(*shape, dt=f32):
    return torch.zeros(shape, dtype=dt)


@pytest.mark.parametrize("args,kw,err", [
    ((z(2, 5, 8, dt=torch.float16), z(2, 5, 8), z(2, 5, 8)), {}, TypeError),
    ((z(2, 5, 8), z(2, 5, 7), z(2, 5, 8)), {}, ValueError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 4, 8)), {}, ValueError),
    ((z(2, 5, 8), z(2, 5, 8), None), {}, ValueError),
    ((z(2, 5, 8), None, z(2, 5, 8)), {}, ValueError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 5, 8)), dict(gates="tied"), ValueError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 5, 8)), dict(gates="scalar"), ValueError),
    ((z(2, 5, 8, dt=bf16), z(2, 5, 8, dt=bf16), z(2, 5, 8, dt=bf16)), {}, TypeError),  # fp32 gates wanted
    ((z(2, 5, 8, dt=bf16), z(2, 5, 8), z(2, 5, 8)), dict(gates="preact"), TypeError),
    ((z(5, 8), z(5, 8), z(5, 8)), {}, ValueError),
    ((z(2, 5, 0), z(2, 5, 0), z(2, 5, 0)), {}, ValueError),
    ((z(2, 8, 5).transpose(1, 2), z(2, 5, 8), z(2, 5, 8)), {}, ValueError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 5, 8), z(1, 8)), {}, ValueError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 5, 8), z(2, 8, dt=bf16)), {}, TypeError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 5, 8)), dict(o=z(2, 5, 9)), ValueError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 5, 8)), dict(h_T=z(8, 2)), ValueError),
    ((z(2, 5, 8), z(2, 5, 8), z(2, 5, 8)), dict(ck=z(2, 2, 8)), ValueError)])
def test_linear_forward_refusals(host_tensors, args, kw, err):
    with pytest.raises(err):
        g.linear_forward(*args, **kw)


def test_linear_other_refusals(host_tensors):
    x, h = z(5, 8), z(2, 8)
    cu = torch.tensor([0, 2, 5], dtype=i32)
    for bad in (dict(cu_seqlens=None), dict(cu_seqlens=cu.long()), dict(cu_seqlens=torch.empty(0, dtype=i32)), dict(h0=z(3, 8))):
        kw = dict(cu_seqlens=cu, h0=h) | bad
        with pytest.raises((ValueError, TypeError)):
            g.linear_forward_varlen(x, x, x, **kw)
        with pytest.raises((ValueError, TypeError)):
            g.linear_backward_varlen(x, x, x, dO=x, **kw)
    with pytest.raises(ValueError):
        g.linear_forward_varlen(z(1, 5, 8), x, x, cu)
    b = z(2, 5, 8)
    for bad in (dict(dO=z(2, 5, 9)), dict(dO=None), dict(dh_T=z(1, 8)), dict(ck=z(2, 1, 9)), dict(grads={"dx": z(2, 5, 9)}),
                dict(grads={"dh0": z(2, 9)}), dict(workspace=z(100))):
        with pytest.raises((ValueError, TypeError)):
            g.linear_backward(b, b, b, h, **(dict(dO=b) | bad))
    s = z(2, 8)
    for args, kw in (((z(3, 8), s, s, h), {}), ((s, s, None, h), {}), ((s, s, s, h), dict(gates="tied")),
                     ((s, s, s, z(8)), {}), ((s, s, s, h), dict(h_out=z(2, 9))), ((s, s, s, h), dict(o=z(2, 1, 8))),
                     ((s, s, s, h), dict(gates="x"))):
        with pytest.raises(ValueError):
            g.linear_step(*args, **kw)


@pytest.mark.parametrize("args,kw,err", [
    ((z(4, 8, dt=torch.float64),), {}, TypeError), ((z(4, 8), z(7)), {}, ValueError), ((z(4, 8), None, z(8, 1)), {}, ValueError),
    ((z(4, 8), z(8), z(8, dt=bf16)), {}, TypeError), ((z(4, 8), z(8, dt=torch.float16)), {}, TypeError),
    ((z(4, 8), z(8), None, z(4, 8, dt=bf16)), {}, TypeError), ((z(4, 8), z(8), None, z(8)), {}, ValueError),
    ((z(4, 0),), {}, ValueError), ((z(8, 4).t(),), {}, ValueError), ((z(4, 8),), dict(kind="group"), ValueError),
    ((z(4, 8),), dict(y=z(4, 9)), ValueError)])
def test_norm_refusals(host_tensors, args, kw, err):
    with pytest.raises(err):
        g.norm_forward(*args, **kw)


def test_norm_backward_refusals(host_tensors):
    x, w = z(4, 8), z(8)
    for dy, kw in ((None, {}), (z(4, 9), {}), (z(4, 8, dt=bf16), {}), (x, dict(grads={"dweight": z(9)})),
                   (x, dict(workspace=z(1000)))):
        with pytest.raises((ValueError, TypeError)):
            g.norm_backward(x, w, w, None, dy, **kw)


def test_cache_refusals(host_tensors):
    c, s, n = z(4, 2, 16, 32, dt=torch.uint8), z(4, 2, 16, dt=torch.uint8), torch.zeros(3, dtype=i32)
    S = z(3, 2, 16, 32)
    for args, kw in (((S, n, c, s), dict(fmt="e5m2")), ((S, n.long(), c, s), {}), ((S, n, c.float(), s), {}),
                     ((S, n, c, z(4, 2, 17, dt=torch.uint8)), {}), ((z(2, 2, 16, 32), n, c, s), {}), ((S.to(bf16), n, c, s), {}),
                     ((S, n, z(4, 32, dt=torch.uint8), z(4, dt=torch.uint8)), {})):
        with pytest.raises((ValueError, TypeError)):
            g.state_cache_store(*args, **kw)
    for kw in (dict(S=z(3, 2, 16, 16)), dict(fmt="x")):
        with pytest.raises(ValueError):
            g.state_cache_load(c, s, n, **kw)


def test_structures_match_the_header():
    """Field sizes as the C compiler lays them out: five or five 32-bit fields, and a 64-bit one first."""
    assert ctypes.sizeof(g.gdn2_linear_desc) == 20 and ctypes.sizeof(g.gdn2_cache_desc) == 20
    assert ctypes.sizeof(g.gdn2_norm_desc) == 32 and g.gdn2_norm_desc.eps.offset == 24


def test_packed_limits_do_not_count_sequences():
    """A packed call's workgroups come from its tokens and channels; B sequences only make B + 1 offsets and B states."""
    queries = (g.gdn2_linear_forward_varlen_workspace_bytes, g.gdn2_linear_backward_varlen_workspace_bytes)
    for d in (lin(B=512, T=65536, D=4096), lin(B=4096, T=8192, D=4096), lin(B=2 ** 24 - 1, T=8192, D=4096),
              lin(B=2 ** 24 - 1, T=64 * (2 ** 24 - 1), D=128), lin(B=2 ** 24 - 1, T=0, D=2 ** 22)):
        assert (d.T == 0) == (queries[0](d) == 0)
        # accepted as a description: the missing offsets are the first thing wrong with the call
        assert fwd_varlen(d, put(fakes(8), _0=0)) == g.GDN2_ERR_NULL_POINTER
        assert g.gdn2_linear_backward_varlen(d, 0, *fakes(11), FAKE - EACH, 1 << 30, 0) == g.GDN2_ERR_NULL_POINTER
        assert fwd(d) == g.GDN2_ERR_UNSUPPORTED and bwd(d) == g.GDN2_ERR_UNSUPPORTED  # as whole sequences: too many
    assert queries[1](lin(B=4096, T=8192, D=4096)) == queries[1](lin(B=1, T=8192, D=4096))
    for d in (lin(B=2 ** 24, T=64), lin(B=1, T=64 * (2 ** 24 - 1) + 1, D=128), lin(B=1, T=64 * (2 ** 24 - 1), D=129),
              lin(B=2 ** 31 - 1, T=1, D=1)):
        assert fwd_varlen(d) == g.GDN2_ERR_UNSUPPORTED and queries[0](d) == queries[1](d) == 0
