"""The norms (gdn2_norm_*) against their 64-bit plain form.

Tolerances. A sum of D values taken by 64 or 256 threads and joined pairwise is
off by at most D_chain = D / 64 + 10 roundings of its terms' sum of magnitudes,
so the mean, the mean square and the two means of the backward are off by at
most K = D_chain * 2^-24 of the mean magnitude of their terms, and r by half
its mean square's. y is a few more roundings (8) of n, z and silu. For dx every
term carries at most (3 K + 16 * 2^-24) of r * (|d| + |xh| mean|d xh| + mean|d|).
The weight's sums over the rows are off by 2^-24 * (rows / 64 + 64) of the sum of
the magnitudes. A bf16 output is off by one more rounding of itself."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def problem(rng, shape, dtype, wtype, bias, gate, weight=True, mean=0.3):
    mk = lambda v, d: torch.tensor(np.asarray(v, np.float32)).to(d).to(DEV)
    D, dt, wt = shape[-1], R.TORCH[dtype], R.TORCH[wtype]
    return dict(x=mk(rng.standard_normal(shape) + mean, dt),
                w=mk(1 + 0.2 * rng.standard_normal(D), wt) if weight else None,
                b=mk(rng.standard_normal(D), wt) if bias else None,
                z=mk(2 * rng.standard_normal(shape), dt) if gate else None, dy=mk(rng.standard_normal(shape), dt))


def bound(name, got, ref, tol, dtype):
    err = np.abs(R.f64(got) - ref)
    tol = tol + (0 if dtype == torch.float32 else R.half(dtype)) * (np.abs(ref) + tol)
    worst = float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0
    print(f"[norm {name}] worst error over its bound {worst:.3f}", flush=True)
    assert np.isfinite(R.f64(got)).all() and worst <= 1.0, name


def check(p, kind, eps, y, gr=None):
    f = {k: R.f64(v) for k, v in p.items()}
    D = f["x"].shape[-1]
    flat = lambda v: None if v is None else v.reshape(-1, D)
    x, z, dy = flat(f["x"]), flat(f["z"]), flat(f["dy"])
    u = R.U32
    K = (D / 64 + 10) * u
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    # the centred value: the mean's error and one rounding; xh: that, r's error, one rounding
    dc = (K * np.abs(x).mean(-1, keepdims=True) if kind == "layer" else 0) + 2 * u * (np.abs(c) + (np.abs(x) if kind == "layer" else 0))
    rel_r = K + (np.abs(c) * dc).mean(-1, keepdims=True) * r * r + 4 * u
    xh = c * r
    dxh = dc * r + np.abs(xh) * (rel_r + 2 * u)
    w, b = 1.0 if f["w"] is None else f["w"], 0.0 if f["b"] is None else f["b"]
    n = xh * w + b
    dn_ = dxh * np.abs(w) + 2 * u * (np.abs(xh * w) + np.abs(n))
    s = np.ones_like(x) if z is None else z * R.sigmoid(z)
    ds = 0 if z is None else 8 * u * (1 + np.abs(z)) * np.abs(s)
    ref = R.norm(x, f["w"], f["b"], z, eps, kind)
    bound("y", flat(y), ref, dn_ * np.abs(s) + np.abs(n) * ds + 2 * u * np.abs(ref), y.dtype)
    if gr is None:
        return
    dx, dw, db, dz = R.norm_grads(x, f["w"], f["b"], z, dy, eps, kind)
    dn = dy * s
    ddn = np.abs(dy) * ds + 2 * u * np.abs(dn)
    d, dd = np.abs(dn * w), ddn * np.abs(w) + 2 * u * np.abs(dn * w)
    mean = lambda v: v.mean(-1, keepdims=True)
    m1 = mean(d * np.abs(xh))
    dm1 = mean(dd * np.abs(xh) + d * dxh) + (K + 4 * u) * m1
    tol = r * (dd + dxh * m1 + np.abs(xh) * dm1 + (mean(dd) + (K + 4 * u) * mean(d) if kind == "layer" else 0))
    tol = tol + (rel_r + 8 * u) * r * (d + np.abs(xh) * m1 + (mean(d) if kind == "layer" else 0))
    bound("dx", flat(gr["dx"]), dx, tol, y.dtype)
    L = (x.shape[0] / 64 + 64) * u
    if p["w"] is not None:
        bound("dweight", gr["dweight"], dw, (L * np.abs(dn * xh) + ddn * np.abs(xh) + np.abs(dn) * dxh).sum(0) + 1e-30,
              p["w"].dtype)
    if p["b"] is not None:
        bound("dbias", gr["dbias"], db, (L * np.abs(dn) + ddn).sum(0) + 1e-30, p["b"].dtype)
    if z is not None:
        sg = R.sigmoid(z)
        ps = sg + np.abs(z) * sg * (1 - sg)
        bound("dgate", flat(gr["dgate"]), dz,
              np.abs(dy) * (dn_ * ps + np.abs(n) * 16 * u * (1 + np.abs(z)) * ps) + 4 * u * np.abs(dz), y.dtype)


SIZES = [(1, 1), (1, 2), (5, 3), (7, 16), (33, 32), (130, 64), (1000, 128), (9, 136), (3, 256), (17, 500), (40, 512),
         (3, 1001), (5, 1024), (6, 2048), (70, 2056), (3, 4096), (2, 4099), (4, 8192), (2, 16384), (1, 16392), (2, 20001)]


@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("kind,bias,gate", [("layer", True, False), ("rms", False, True), ("layer", True, True),
                                            ("rms", False, False)])
@pytest.mark.parametrize("rows,D", SIZES)
def test_forward_and_gradients(rows, D, kind, bias, gate, dtype, wtype):
    p = problem(np.random.default_rng(rows * 7 + D), (rows, D), dtype, wtype, bias, gate)
    y = g.norm_forward(p["x"], p["w"], p["b"], p["z"], eps=1e-5, kind=kind)
    gr = g.norm_backward(p["x"], p["w"], p["b"], p["z"], p["dy"], eps=1e-5, kind=kind)
    torch.cuda.synchronize()
    check(p, kind, float(np.float32(1e-5)), y, gr)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("shape", [(2, 50, 4, 128), (3, 7, 40)])
def test_any_leading_shape_without_weights(shape, kind):
    p = problem(np.random.default_rng(1), shape, "bf16", "f32", False, False, weight=False)
    y = g.norm_forward(p["x"], kind=kind)
    gr = g.norm_backward(p["x"], None, None, None, p["dy"], kind=kind)
    torch.cuda.synchronize()
    assert y.shape == p["x"].shape and gr["dweight"] is None and gr["dbias"] is None and gr["dgate"] is None
    check(p, kind, float(np.float32(1e-5)), y, gr)


@pytest.mark.parametrize("rows,D", [(5, 128), (4, 2048), (3, 1001)])
def test_constant_rows_and_large_offsets(rows, D):
    """A constant row normalises to the bias; a common offset of 1000 costs no
    more than the offset's own rounding (the mean is taken before the squares)."""
    p = problem(np.random.default_rng(2), (rows, D), "f32", "f32", True, False)
    x = p["x"].clone()
    x[0] = 3.25
    y = g.norm_forward(x, p["w"], p["b"])
    torch.cuda.synchronize()
    # the mean of D equal values: off by at most (D / 64 + 10) roundings, over sqrt(eps)
    assert ((y[0] - p["b"]).abs() <= (D / 64 + 10) * R.U32 * 3.25 / 1e-5 ** 0.5 * p["w"].abs() + 1e-6).all()
    p["x"] = p["x"] + 1000.0
    y = g.norm_forward(p["x"], p["w"], p["b"])
    check(p, "layer", float(np.float32(1e-5)), y)


@pytest.mark.parametrize("D", [64, 500, 2048, 1001])
def test_a_bad_row_stays_alone(D):
    p = problem(np.random.default_rng(4), (40, D), "bf16", "f32", True, True)
    good = {k: v.clone() if k in ("x", "z", "dy") else v for k, v in p.items()}
    y0 = g.norm_forward(good["x"], p["w"], p["b"], good["z"])
    d0 = g.norm_backward(good["x"], p["w"], p["b"], good["z"], good["dy"])
    p["x"][7, 3], p["x"][21, 0] = float("nan"), float("inf")
    y = g.norm_forward(p["x"], p["w"], p["b"], p["z"])
    gr = g.norm_backward(p["x"], p["w"], p["b"], p["z"], p["dy"])
    torch.cuda.synchronize()
    keep = [i for i in range(40) if i not in (7, 21)]
    assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[7]).all()
    assert torch.equal(gr["dx"][keep], d0["dx"][keep]) and torch.equal(gr["dgate"][keep], d0["dgate"][keep])


def test_no_rows_and_parts_not_wanted():
    e = torch.empty(0, 64, device=DEV)
    w, b = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    assert g.norm_forward(e, w, b).shape == (0, 64)
    gr = g.norm_backward(e, w, b, None, e)
    torch.cuda.synchronize()
    assert (gr["dweight"] == 0).all() and (gr["dbias"] == 0).all()
    p = problem(np.random.default_rng(6), (300, 96), "bf16", "f32", True, True)
    full = g.norm_backward(p["x"], p["w"], p["b"], p["z"], p["dy"])
    part = g.norm_backward(p["x"], p["w"], p["b"], p["z"], p["dy"], want_params=False, want_dgate=False)
    assert part["dweight"] is None and part["dbias"] is None and part["dgate"] is None
    assert torch.equal(full["dx"], part["dx"])


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("D", [24, 37])
def test_gradients_against_differences(D, kind):
    """Along random directions against central differences of the 64-bit plain
    form (their own error: 1e-10 of third derivatives of order 1e3)."""
    rng = np.random.default_rng(8)
    p = problem(rng, (30, D), "f32", "f32", True, True)
    leaf = {k: p[k].clone().requires_grad_() for k in ("x", "w", "b", "z")}
    y = g.norm(leaf["x"], leaf["w"], leaf["b"], leaf["z"], eps=1e-3, kind=kind)
    grads = dict(zip(leaf, torch.autograd.grad(y, list(leaf.values()), p["dy"])))
    f = {k: R.f64(v) for k, v in p.items()}
    loss = lambda q: (R.norm(q["x"], q["w"], q["b"], q["z"], float(np.float32(1e-3)), kind) * f["dy"]).sum()
    for k in leaf:
        v = rng.standard_normal(f[k].shape)
        num = (loss(dict(f, **{k: f[k] + 1e-5 * v})) - loss(dict(f, **{k: f[k] - 1e-5 * v}))) / 2e-5
        got = (R.f64(grads[k]) * v).sum()
        print(f"[norm differences {kind} {k}] {got:.8g} {num:.8g}", flush=True)
        # at most 64 roundings of each gradient value
        assert abs(got - num) <= 64 * R.U32 * np.abs(R.f64(grads[k])).max() * np.abs(v).sum() + 1e-6 * (1 + abs(num))


def test_a_replayed_graph_and_repeatability():
    p = problem(np.random.default_rng(9), (5000, 128), "bf16", "f32", True, True)
    args = (p["x"], p["w"], p["b"], p["z"])
    y, gr = g.norm_forward(*args), g.norm_backward(*args, p["dy"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = g.norm_forward(*args), g.norm_backward(*args, p["dy"])
    for i in range(4):
        for t in (y2, *g2.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(gr[k], g2[k]) for k in gr), i
        again = g.norm_backward(*args, p["dy"])
        torch.cuda.synchronize()
        assert all(torch.equal(gr[k], again[k]) for k in gr), i


def test_offsets_past_32_bits():
    rows, D = (1 << 31) // 2048 + 5, 2048
    x = torch.zeros(rows, D, dtype=torch.bfloat16, device=DEV)
    p = problem(np.random.default_rng(10), (4, D), "bf16", "f32", False, False)
    x[-4:] = p["x"]
    y = g.norm_forward(x, p["w"])
    dy = torch.zeros_like(x)
    dy[-4:] = p["dy"]
    gr = g.norm_backward(x, p["w"], None, None, dy)
    torch.cuda.synchronize()
    assert (y[:-4] == 0).all() and (gr["dx"][:-4] == 0).all()
    check(p, "layer", float(np.float32(1e-5)), y[-4:], dict(gr, dx=gr["dx"][-4:]))


def closed(z):
    """The gate as the header defines it: below -87 its factor silu(gate) is 0 (1.5e-36 at -87), and so is its derivative."""
    return torch.where(z.double() < -87.0, torch.full_like(z, -1e4, dtype=torch.float64), z.double())


# one row plan each: lanes of a wave with wide, 8-byte and single loads, workgroups with one, two and four pieces a
# lane, and rows past the registers with vectors and single values
FAR = [(9, 128), (9, 500), (9, 137), (6, 1024), (6, 2052), (5, 1001), (3, 8192), (3, 16392), (3, 5001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,bias", [("layer", True), ("rms", False)])
@pytest.mark.parametrize("rows,D", FAR)
def test_closed_gates(rows, D, kind, bias, dtype):
    """Gates far below 0, the type's lowest value and -inf among them, close their channels: nothing of them is left
    in the result or in any gradient, and the other channels are what they are without them."""
    p = problem(np.random.default_rng(rows + D), (rows, D), dtype, "f32", bias, True)
    low = torch.finfo(R.TORCH[dtype]).min
    far = torch.tensor([-70.0, -88.0, -100.0, -104.0, -1e4, -1e30, -1e36, low, -float("inf")], device=DEV)
    at = torch.arange(0, D, 5, device=DEV)
    p["z"][:, at] = far[torch.arange(len(at), device=DEV) % len(far)].to(p["z"].dtype)
    p["z"][1] = low  # a row whose gate leaves nothing
    y = g.norm_forward(p["x"], p["w"], p["b"], p["z"], kind=kind)
    gr = g.norm_backward(p["x"], p["w"], p["b"], p["z"], p["dy"], kind=kind)
    torch.cuda.synchronize()
    shut = p["z"].float() < -87.0
    assert (y[shut] == 0).all() and (gr["dgate"][shut] == 0).all()
    assert (y[1] == 0).all() and (gr["dx"][1] == 0).all() and (gr["dgate"][1] == 0).all()
    check(dict(p, z=closed(p["z"])), kind, float(np.float32(1e-5)), y, gr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [128, 137, 1024, 1001, 16392, 5001])
def test_open_gates(D, dtype):
    """Gates far above 0: silu(gate) is the gate and its derivative 1, for +inf too."""
    p = problem(np.random.default_rng(D), (3, D), dtype, "f32", True, True)
    for i, v in enumerate((100.0, 1e30, float("inf"))):
        p["z"][i, ::7] = v
    y = g.norm_forward(p["x"], p["w"], p["b"], p["z"])
    gr = g.norm_backward(p["x"], p["w"], p["b"], p["z"], p["dy"])
    torch.cuda.synchronize()
    n = R.norm(R.f64(p["x"]), R.f64(p["w"]), R.f64(p["b"]), None, float(np.float32(1e-5)), "layer")[:, ::7]
    # n: its mean's, root's and own roundings as in check, at most 4 K of its terms' size, 1 + |w| + |b| + |n| here
    tol = 4 * (D / 64 + 10) * R.U32 * (1 + np.abs(n) + np.abs(R.f64(p["w"]))[::7] + np.abs(R.f64(p["b"]))[::7])
    half, dy = 0.0 if dtype == "f32" else R.half(R.TORCH[dtype]), R.f64(p["dy"])[:, ::7]
    assert (np.abs(R.f64(gr["dgate"])[:, ::7] - dy * n) <= np.abs(dy) * tol + (half + 4 * R.U32) * np.abs(dy) * (np.abs(n) + tol)).all()
    z = R.f64(p["z"])[:2, ::7]
    assert (np.abs(R.f64(y)[:2, ::7] - n[:2] * z) <= np.abs(z) * (tol + (half + 4 * R.U32) * (np.abs(n) + tol))[:2]).all()
    sure = np.abs(n[2]) > tol[2]
    assert (R.f64(y)[2, ::7][sure] == (np.sign(n[2]) * np.inf)[sure]).all()
