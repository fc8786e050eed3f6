"""Host checks of the attention layer's operators: every refused call returns its
status before any HIP call (made-up addresses that are never read), and the torch
conveniences refuse what would be read or written out of its bounds before the
library is reached."""
import ctypes

import pytest
import torch

import gated_delta_rule_83_amd as g

FAKE, EACH = 1 << 40, 1 << 36  # distinct made-up buffers, EACH bytes apart
NULL, SHAPE, UNSUPPORTED, DTYPE, WORKSPACE, ALIAS = (g.GDN2_ERR_NULL_POINTER, g.GDN2_ERR_BAD_SHAPE, g.GDN2_ERR_UNSUPPORTED,
                                                     g.GDN2_ERR_BAD_DTYPE, g.GDN2_ERR_WORKSPACE, g.GDN2_ERR_ALIAS)
WS = FAKE - EACH
INF, NAN = float("inf"), float("nan")


def fakes(n):
    return [FAKE + i * EACH for i in range(n)]


def put(p, **at):
    p = list(p)
    for k, v in at.items():
        p[int(k[1:])] = v
    return p


# ------------------------------------------------------------------ rotary
def rot(tokens=100, H_q=4, H_k=2, d=64, rot=64, norm=1, pairs=0, dtype=1, wdtype=0, eps=1e-6, sq=0, sk=0):
    return g.gdn2_rotary_desc(tokens, H_q, H_k, d, rot, norm, pairs, dtype, wdtype, eps, sq, sk)


BAD_ROTARY = [(None, NULL), (rot(dtype=2), DTYPE), (rot(wdtype=-1), DTYPE), (rot(tokens=-1), SHAPE), (rot(H_q=-1), SHAPE),
              (rot(H_k=-1), SHAPE), (rot(d=0), SHAPE), (rot(rot=-2), SHAPE), (rot(rot=66), SHAPE), (rot(eps=-1.0), SHAPE),
              (rot(eps=NAN), SHAPE), (rot(eps=INF), SHAPE), (rot(d=65, rot=64), UNSUPPORTED), (rot(rot=63), UNSUPPORTED),
              (rot(d=1026), UNSUPPORTED), (rot(pairs=2), UNSUPPORTED), (rot(pairs=-1), UNSUPPORTED),
              (rot(tokens=2 ** 31), UNSUPPORTED), (rot(H_q=2 ** 17), UNSUPPORTED), (rot(sq=2 ** 22 + 64), UNSUPPORTED),
              (rot(sq=255), SHAPE), (rot(sk=64), SHAPE), (rot(sq=-256), SHAPE)]


@pytest.mark.parametrize("desc,status", BAD_ROTARY)
def test_rotary_descriptions(desc, status):
    assert g.gdn2_rotary_forward(desc, *fakes(8)) == status
    assert g.gdn2_rotary_backward(desc, *fakes(12), WS, 1 << 30) == status
    assert g.gdn2_rotary_backward_workspace_bytes(desc) == 0


def test_rotary_pointers():
    f = fakes(8)  # q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out
    fwd = lambda p, d=None: g.gdn2_rotary_forward(d or rot(), *p)  # noqa: E731
    for i in (0, 1, 4, 5, 6, 7):
        assert fwd(put(f, **{f"_{i}": 0})) == NULL, i
    for i, off in ((0, 1), (1, 1), (2, 2), (3, 2), (4, 2), (5, 2), (6, 1), (7, 1)):
        assert fwd(put(f, **{f"_{i}": f[i] + off})) == SHAPE, i
    for out in (6, 7):
        for i in range(6):
            assert fwd(put(f, **{f"_{out}": f[i]})) == ALIAS, (out, i)
    assert fwd(put(f, _7=f[6])) == ALIAS
    # a view's reach counts: k behind q in one fused projection of 512 values, the result in between
    assert fwd(put(f, _1=f[0] + 512, _6=f[0] + 2048), rot(sq=512, sk=512)) == ALIAS
    assert fwd([0] * 8, rot(tokens=0)) == g.GDN2_OK and fwd([0] * 8, rot(H_q=0, H_k=0)) == g.GDN2_OK
    b = fakes(12)  # q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, dq, dk, dq_weight, dk_weight
    bwd = lambda p, ws=1 << 30, at=WS: g.gdn2_rotary_backward(rot(), *p, at, ws)  # noqa: E731
    for i in (0, 1, 4, 5, 6, 7, 8, 9, 2, 3):
        assert bwd(put(b, **{f"_{i}": 0})) == NULL, i
    need = g.gdn2_rotary_backward_workspace_bytes(rot())
    assert need > 0 and bwd(b, need - 1) == WORKSPACE and bwd(b, need, 0) == WORKSPACE
    assert bwd(b, need, WS + 4) == SHAPE and bwd(b, need, b[0]) == ALIAS
    for out in (8, 9, 10, 11):
        for i in range(8):
            assert bwd(put(b, **{f"_{out}": b[i]})) == ALIAS, (out, i)


# ------------------------------------------------------------------ attention
def att(B=2, T_q=100, T_k=120, H=4, H_kv=2, d=64, causal=1, window=0, dtype=1, scale=0.1, sq=0, sk=0, sv=0):
    return g.gdn2_attention_desc(B, T_q, T_k, H, H_kv, d, causal, window, dtype, scale, sq, sk, sv)


BAD_ATTENTION = [(None, NULL), (att(dtype=2), DTYPE), (att(B=-1), SHAPE), (att(T_q=-1), SHAPE), (att(T_k=-1), SHAPE),
                 (att(H=0), SHAPE), (att(H_kv=0), SHAPE), (att(H=5), SHAPE), (att(window=-1), SHAPE), (att(scale=0.0), SHAPE),
                 (att(scale=-1.0), SHAPE), (att(scale=NAN), SHAPE), (att(scale=INF), SHAPE), (att(d=32), UNSUPPORTED),
                 (att(d=96), UNSUPPORTED), (att(d=256), UNSUPPORTED), (att(window=5, causal=0), UNSUPPORTED),
                 (att(sq=255), SHAPE), (att(sq=260), SHAPE), (att(sk=64), SHAPE), (att(sv=132), SHAPE), (att(sk=-128), SHAPE),
                 (att(sq=2 ** 22 + 64), UNSUPPORTED), (att(H=2 ** 17, H_kv=1), UNSUPPORTED), (att(T_q=2 ** 31 - 1), UNSUPPORTED),
                 (att(T_k=2 ** 31 - 1), UNSUPPORTED), (att(B=2 ** 24), UNSUPPORTED)]


@pytest.mark.parametrize("desc,status", BAD_ATTENTION)
def test_attention_descriptions(desc, status):
    assert g.gdn2_attention_forward(desc, *fakes(5)) == status
    assert g.gdn2_attention_forward_varlen(desc, *fakes(7)) == status
    assert g.gdn2_attention_backward(desc, *fakes(9), WS, 1 << 34) == status
    assert g.gdn2_attention_backward_varlen(desc, *fakes(11), WS, 1 << 34) == status
    assert g.gdn2_attention_backward_workspace_bytes(desc) == g.gdn2_attention_backward_varlen_workspace_bytes(desc) == 0


def test_attention_limits_count_blocks():
    for T in (dict(T_q=2 ** 31 - 257, T_k=1), dict(T_k=2 ** 31 - 257, T_q=1)):
        assert g.gdn2_attention_forward(att(B=1, H=1, H_kv=1, **T), *[0] * 5) == NULL  # 2^24 - 2 blocks: fine
        assert g.gdn2_attention_forward(att(B=1, H=2, H_kv=1, **T), *[0] * 5) == UNSUPPORTED
    # two threads for each of the forward's in the backward
    assert g.gdn2_attention_backward(att(B=1, H=1, H_kv=1, T_q=2 ** 30 - 256, T_k=1), *[0] * 9, WS, 1 << 60) == NULL
    assert g.gdn2_attention_backward(att(B=1, H=1, H_kv=1, T_q=1, T_k=2 ** 30 + 1), *[0] * 9, WS, 1 << 60) == UNSUPPORTED
    # packed: a block of room a sequence
    assert g.gdn2_attention_forward_varlen(att(B=2 ** 22, H=3, H_kv=1), *[0] * 7) == NULL
    assert g.gdn2_attention_forward_varlen(att(B=2 ** 22, H=4, H_kv=1), *[0] * 7) == UNSUPPORTED


def test_attention_pointers():
    f = fakes(5)  # q, k, v, o, lse
    fwd = lambda p, d=None: g.gdn2_attention_forward(d or att(), *p)  # noqa: E731
    for i in range(4):
        assert fwd(put(f, **{f"_{i}": 0})) == NULL, i
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 8), (4, 2)):
        assert fwd(put(f, **{f"_{i}": f[i] + off})) == SHAPE, i
    for out in (3, 4):
        for i in range(3):
            assert fwd(put(f, **{f"_{out}": f[i] + 64})) == ALIAS, (out, i)
    assert fwd(put(f, _4=f[3])) == ALIAS
    assert fwd(put(f, _3=f[0] + 1024), att(sq=4096)) == ALIAS  # between a view's tokens: within its reach
    for d in (att(B=0), att(T_q=0)):
        assert fwd([0] * 5, d) == g.GDN2_OK
    v = fakes(7)
    for i in range(6):
        assert g.gdn2_attention_forward_varlen(att(), *put(v, **{f"_{i}": 0})) == NULL, i
    assert g.gdn2_attention_forward_varlen(att(), *put(v, _0=v[0] + 2)) == SHAPE
    assert g.gdn2_attention_forward_varlen(att(), *put(v, _5=v[1])) == ALIAS


def test_attention_backward_pointers_and_workspace():
    f = fakes(9)  # q, k, v, o, lse, dO, dq, dk, dv
    need = g.gdn2_attention_backward_workspace_bytes(att())
    bwd = lambda p, ws=need, at=WS, d=None: g.gdn2_attention_backward(d or att(), *p, at, ws)  # noqa: E731
    for i in range(9):
        assert bwd(put(f, **{f"_{i}": 0})) == NULL, i
    for i in (0, 1, 2, 3, 5, 6, 7, 8):
        assert bwd(put(f, **{f"_{i}": f[i] + 8})) == SHAPE, i
    assert bwd(f, need - 1) == WORKSPACE and bwd(f, need, 0) == WORKSPACE and bwd(f, need, WS + 8) == SHAPE
    for out in (6, 7, 8):
        for i in range(6):
            assert bwd(put(f, **{f"_{out}": f[i]})) == ALIAS, (out, i)
    assert bwd(put(f, _7=f[8])) == ALIAS and bwd(f, need, f[1]) == ALIAS
    # lse and delta of every query, and few key blocks: a share of dk and dv for each query head
    assert need >= 2 * 2 * 4 * 100 * 4 + 2 * 2 * (2 * 120 * 2 * 64) * 4
    assert bwd([0] * 9, 0, 0, att(T_q=0, T_k=0)) == g.GDN2_OK
    # queries without keys and keys without queries still have gradients
    assert bwd([0] * 9, 1 << 30, WS, att(T_k=0)) == NULL and bwd([0] * 9, 1 << 30, WS, att(T_q=0)) == NULL
    v = fakes(11)
    for i in (0, 1):
        assert g.gdn2_attention_backward_varlen(att(), *put(v, **{f"_{i}": 0}), WS, 1 << 34) == NULL
    assert g.gdn2_attention_backward_varlen(att(), *put(v, _8=v[0]), WS, 1 << 34) == ALIAS


# ------------------------------------------------------------------ decode and cache
def dec(N=4, H=8, H_kv=2, d=64, P=100, page=16, M=200, window=0, dtype=1, scale=0.1):
    return g.gdn2_attention_decode_desc(N, H, H_kv, d, P, page, M, window, dtype, scale)


BAD_DECODE = [(None, NULL), (dec(dtype=3), DTYPE), (dec(N=-1), SHAPE), (dec(P=-1), SHAPE), (dec(M=-1), SHAPE), (dec(H=0), SHAPE),
              (dec(H_kv=0), SHAPE), (dec(H=9), SHAPE), (dec(window=-1), SHAPE), (dec(page=0), SHAPE), (dec(scale=0.0), SHAPE),
              (dec(scale=NAN), SHAPE), (dec(d=32), UNSUPPORTED), (dec(page=48), UNSUPPORTED), (dec(M=2 ** 20, page=2048), UNSUPPORTED),
              (dec(N=2 ** 22), UNSUPPORTED), (dec(N=2 ** 19, M=1), UNSUPPORTED)]


@pytest.mark.parametrize("desc,status", BAD_DECODE)
def test_decode_descriptions(desc, status):
    assert g.gdn2_attention_decode(desc, *fakes(6), WS, 1 << 34) == status
    assert g.gdn2_attention_decode_workspace_bytes(desc) == 0


def test_decode_pointers_and_workspace():
    f = fakes(6)  # q, k_cache, v_cache, pages, lengths, o
    need = g.gdn2_attention_decode_workspace_bytes(dec())
    run = lambda p, ws=need, at=WS, d=None: g.gdn2_attention_decode(d or dec(), *p, at, ws)  # noqa: E731
    assert need >= 4 * 8 * 2 * 66 * 4
    for i in range(6):
        assert run(put(f, **{f"_{i}": 0})) == NULL, i
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 2), (4, 2), (5, 8)):
        assert run(put(f, **{f"_{i}": f[i] + off})) == SHAPE, i
    for i in range(5):
        assert run(put(f, _5=f[i])) == ALIAS and run(f, need, f[i]) == ALIAS, i
    assert run(f, need - 1) == WORKSPACE and run(f, need, 0) == WORKSPACE and run(f, need, WS + 8) == SHAPE
    assert run([0] * 6, 0, 0, dec(N=0)) == g.GDN2_OK
    # up to 512 keys, of the table or of the window, are one span: no workspace
    assert g.gdn2_attention_decode_workspace_bytes(dec(M=32)) == 0 and g.gdn2_attention_decode_workspace_bytes(dec(window=400)) == 0
    # spans grow with the table, so that there are 1024 at most
    most = g.gdn2_attention_decode_workspace_bytes(dec(N=1, M=2 ** 26))
    assert 0 < most <= 8 * 1024 * 66 * 4


def sto(N=3, T=50, H_kv=2, d=64, P=100, page=16, M=20, dtype=1, sk=0, sv=0):
    return g.gdn2_kv_cache_desc(N, T, H_kv, d, P, page, M, dtype, sk, sv)


@pytest.mark.parametrize("desc,status", [
    (None, NULL), (sto(dtype=2), DTYPE), (sto(N=-1), SHAPE), (sto(T=-1), SHAPE), (sto(P=-1), SHAPE), (sto(M=-1), SHAPE),
    (sto(H_kv=0), SHAPE), (sto(page=0), SHAPE), (sto(sk=64), SHAPE), (sto(sv=132), SHAPE), (sto(d=48), UNSUPPORTED),
    (sto(page=3), UNSUPPORTED), (sto(M=2 ** 21, page=1024), UNSUPPORTED), (sto(H_kv=2 ** 17), UNSUPPORTED),
    (sto(T=2 ** 31 - 1), UNSUPPORTED), (sto(N=2 ** 31 - 1), UNSUPPORTED)])
def test_store_descriptions(desc, status):
    assert g.gdn2_kv_cache_store(desc, *fakes(7)) == status


def test_store_pointers():
    f = fakes(7)  # cu_seqlens, k, v, pages, lengths, k_cache, v_cache
    assert g.gdn2_kv_cache_store(sto(), 0, *f[1:]) == SHAPE  # one token a sequence: T = N
    for i in range(1, 7):
        assert g.gdn2_kv_cache_store(sto(), *put(f, **{f"_{i}": 0})) == NULL, i
    for i, off in ((0, 2), (1, 8), (2, 8), (3, 2), (4, 2), (5, 8), (6, 8)):
        assert g.gdn2_kv_cache_store(sto(), *put(f, **{f"_{i}": f[i] + off})) == SHAPE, i
    for out in (5, 6):
        for i in range(5):
            assert g.gdn2_kv_cache_store(sto(), *put(f, **{f"_{out}": f[i]})) == ALIAS, (out, i)
    assert g.gdn2_kv_cache_store(sto(), *put(f, _6=f[5])) == ALIAS
    for d in (sto(N=0), sto(T=0), sto(P=0), sto(M=0)):
        assert g.gdn2_kv_cache_store(d, f[0], *[0] * 6) == g.GDN2_OK


def test_structures_match_the_header():
    """Field sizes as the C compiler lays them out: 64-bit fields 8-byte aligned, behind the 32-bit ones."""
    assert ctypes.sizeof(g.gdn2_rotary_desc) == 64 and g.gdn2_rotary_desc.eps.offset == 40 and g.gdn2_rotary_desc.stride_q.offset == 48
    assert ctypes.sizeof(g.gdn2_attention_desc) == 64 and g.gdn2_attention_desc.scale.offset == 36
    assert g.gdn2_attention_desc.stride_q.offset == 40 and ctypes.sizeof(g.gdn2_attention_decode_desc) == 40
    assert ctypes.sizeof(g.gdn2_kv_cache_desc) == 48 and g.gdn2_kv_cache_desc.stride_k.offset == 32


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

    for mod in (g.attention_ops, g.rotary_ops):
        monkeypatch.setattr(mod, "launch_on", here)
        for nm in g.EXPORTED:
            if hasattr(mod, nm) and not nm.endswith("_bytes"):
                monkeypatch.setattr(mod, nm, refuse)


f32, bf16, i32, f16 = torch.float32, torch.bfloat16, torch.int32, torch.float16


def z(*shape, dt=f32):
    return torch.zeros(shape, dtype=dt)


Q, K, P5, F = z(5, 4, 64), z(5, 2, 64), z(5, dt=i32), z(32)


@pytest.mark.parametrize("args,kw", [
    ((Q.to(f16), K, P5, F), {}), ((Q[0], K[0], P5, F), {}), ((Q, z(6, 2, 64), P5, F), {}), ((Q, z(5, 2, 32), P5, F), {}),
    ((Q, K.to(bf16), P5, F), {}), ((Q, K, P5.long(), F), {}), ((Q, K, z(6, dt=i32), F), {}), ((Q, K, None, F), {}),
    ((Q, K, P5, None), {}), ((Q, K, P5, F.double()), {}), ((Q, K, P5, F, z(63)), {}), ((Q, K, P5, F, z(64), z(64, dt=bf16)), {}),
    ((Q, None, P5, F, None, z(64)), {}), ((Q, K, P5, F), dict(pairs="thirds")), ((Q, K, P5, F), dict(q_out=z(5, 4, 63))),
    ((Q, K, P5, F), dict(k_out=z(5, 2, 64, dt=bf16))), ((Q.transpose(1, 2), K, P5, F), {}), ((Q[:, :, ::2], K, P5, F), {}),
    ((Q.expand(5, 4, 64)[:, ::2], K, P5, F), {}), ((Q[:1].expand(5, 4, 64), K, P5, F), {}),
    ((z(2, 6, 4, 64)[:, :5], z(2, 5, 2, 64), z(2, 5, dt=i32), F), {})])
def test_rotary_refusals(host_tensors, args, kw):
    with pytest.raises((ValueError, TypeError)):
        g.rotary_forward(*args, **kw)


def test_rotary_backward_refusals(host_tensors):
    w = z(64)
    for gq, gk, kw in ((None, K, {}), (Q, None, {}), (z(5, 4, 63), K, {}), (Q.to(bf16), K, {}), (Q, K, dict(grads={"dq": z(5, 4, 1)})),
                       (Q, K, dict(grads={"dk_weight": z(3)})), (Q, K, dict(workspace=z(100)))):
        with pytest.raises((ValueError, TypeError)):
            g.rotary_backward(Q, K, P5, F, w, w, gq, gk, **kw)


q4, k4 = z(2, 7, 4, 64), z(2, 9, 2, 64)


@pytest.mark.parametrize("args,kw", [
    ((q4.to(f16), k4, k4), {}), ((q4, k4, k4.to(bf16)), {}), ((q4, k4, z(2, 8, 2, 64)), {}), ((q4, z(1, 9, 2, 64), k4), {}),
    ((q4, z(2, 9, 3, 64), z(2, 9, 3, 64)), {}), ((q4, z(2, 9, 2, 32), z(2, 9, 2, 32)), {}), ((q4[0], k4[0], k4[0]), {}),
    ((q4, k4, k4), dict(o=z(2, 7, 4, 63))), ((q4, k4, k4), dict(lse=z(2, 7, 4))), ((q4, k4, k4), dict(lse=z(2, 4, 7, dt=bf16))),
    ((q4.transpose(1, 2).contiguous().transpose(1, 2), k4, k4), {}), ((q4, z(2, 9, 2, 128)[..., ::2], k4), {}),
    ((z(3, 7, 4, 64)[::2], z(2, 9, 2, 64)[:, :8], z(2, 9, 2, 64)[:, :8]), {}), ((q4, k4, z(2, 9, 0, 64)), {})])
def test_attention_refusals(host_tensors, args, kw):
    with pytest.raises((ValueError, TypeError)):
        g.attention_forward(*args, **kw)


def test_attention_varlen_and_backward_refusals(host_tensors):
    q, k, cu = z(7, 4, 64), z(7, 2, 64), torch.tensor([0, 3, 7], dtype=i32)
    for args, kw in (((q, k, k, None), {}), ((q, k, k, cu.long()), {}), ((q, k, k, torch.empty(0, dtype=i32)), {}),
                     ((q, k, k, cu, cu[:2].contiguous()), {}), ((q[None], k[None], k[None], cu), {}),
                     ((q, k, k, cu), dict(lse=z(7, 4)))):
        with pytest.raises((ValueError, TypeError)):
            g.attention_forward_varlen(*args, **kw)
    lse = z(2, 4, 7)
    for args, kw in (((None, lse, q4), {}), ((q4, None, q4), {}), ((q4, lse, None), {}), ((q4, z(2, 7, 4), q4), {}),
                     ((q4, lse, q4.to(bf16)), {}), ((q4, lse, q4.expand(2, 7, 4, 64).transpose(0, 1)), {}),
                     ((q4, lse, q4), dict(grads={"dk": z(2, 9, 2, 63)})), ((q4, lse, q4), dict(workspace=z(100)))):
        with pytest.raises((ValueError, TypeError)):
            g.attention_backward(q4, k4, k4, *args, **kw)


def test_cache_refusals(host_tensors):
    kc, pages, ln = z(10, 2, 16, 64), z(3, 4, dt=i32), z(3, dt=i32)
    q, k = z(3, 1, 4, 64), z(3, 1, 2, 64)
    for args, kw in (((q, kc, z(10, 2, 16, 32), pages, ln), {}), ((q, kc.to(bf16), kc, pages, ln), {}), ((q, kc, kc, pages.long(), ln), {}),
                     ((q, kc, kc, pages, z(4, dt=i32)), {}), ((q, kc, kc, pages[0], ln), {}), ((q, kc[0], kc[0], pages, ln), {}),
                     ((z(3, 4, 64), kc, kc, pages, ln), {}), ((z(2, 1, 4, 64), kc, kc, pages, ln), {}), ((z(3, 1, 5, 64), kc, kc, pages, ln), {}),
                     ((q.to(bf16), kc, kc, pages, ln), {}), ((q, kc, kc, pages, ln), dict(o=z(3, 1, 4, 63))),
                     ((q, kc.transpose(1, 2), kc.transpose(1, 2), pages, ln), {})):
        with pytest.raises((ValueError, TypeError)):
            g.attention_decode(*args, **kw)
    cu = torch.tensor([0, 1, 4, 6], dtype=i32)
    t = z(6, 2, 64)
    for args, kw in (((k, z(3, 1, 2, 32), pages, ln, kc, kc), {}), ((t, t, pages, ln, kc, kc), {}), ((k.to(bf16), k, pages, ln, kc, kc), {}),
                     ((t, t, pages, ln, kc, kc), dict(cu_seqlens=cu[:3].contiguous())), ((t, t, pages, ln, kc, kc), dict(cu_seqlens=cu.long())),
                     ((t, z(5, 2, 64), pages, ln, kc, kc), dict(cu_seqlens=cu)), ((k, k, pages, z(2, dt=i32), kc, kc), {})):
        with pytest.raises((ValueError, TypeError)):
            g.kv_cache_store(*args, **kw)

