"""Cases, plain forms and 64-bit definitions of the recurrent layer's neighbours of the delta rule.

Three operators:

  linear   the gated linear recurrence h_t = a_t * h_(t-1) + b_t * x_t, channel by channel: whole sequences, packed
           sequences of different lengths, single tokens, and the gradients of the first two;
  norm     layer norm and root-mean-square norm over the last axis, optionally times silu(gate), and their gradients;
  cache    recurrent states written to a cache in 8 bits, one power-of-two scale a row, and read back.

`run` computes a case in elementary torch operations, or with the package's own operators where `own` is true.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one 1.3B-class layer's tokens, the per-channel gates as a model hands them over
        dict(name="linear_layer", op="linear", B=8, T=4096, D=2048, dtype="bf16", gates="channel", train=False),
        # one long document: few channels, many tokens, gates still as pre-activations
        dict(name="linear_long", op="linear", B=1, T=65536, D=2048, dtype="bf16", gates="preact", train=False),
        # a training step of the same layer
        dict(name="linear_train", op="linear", B=8, T=4096, D=2048, dtype="bf16", gates="preact", train=True),
        # a training step of one ragged sequence in full precision, the input gate tied to the decay
        dict(name="linear_train_f32", op="linear", B=1, T=16411, D=1028, dtype="f32", gates="tied", train=True),
        # a prefill batch as a server packs it: sequences of all lengths, some empty
        dict(name="linear_packed", op="packed", N=61, T=32768, D=4096, dtype="bf16", gates="channel", train=False),
        # one token for each of 256 sequences
        dict(name="linear_step", op="step", N=256, D=2048, dtype="bf16", gates="preact"),
        # the mixing layer's output, head by head, with its output gate
        dict(name="norm_heads", op="norm", rows=524288, D=128, dtype="bf16", wtype="f32", kind="rms", bias=False,
             gate=True, train=False),
        # a training step of the norm before a layer
        dict(name="norm_train", op="norm", rows=32768, D=2048, dtype="bf16", wtype="f32", kind="layer", bias=True,
             gate=False, train=True),
        # an odd width in full precision
        dict(name="norm_train_odd", op="norm", rows=4099, D=1001, dtype="f32", wtype="f32", kind="layer", bias=True,
             gate=False, train=True),
        # one token for each of 256 sequences
        dict(name="norm_step", op="norm", rows=256, D=2048, dtype="bf16", wtype="bf16", kind="rms", bias=False,
             gate=True, train=False),
        # the delta rule's states of a full decode batch, put aside and taken back
        dict(name="cache_batch", op="cache", N=256, P=300, H=16, dk=128, dv=128, fmt="e4m3", store=True),
        # five requests that resume from a cached prefix
        dict(name="cache_resume", op="cache", N=5, P=64, H=32, dk=128, dv=128, fmt="int8", store=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _width(rng, lo, hi):
    """A width spread over its logarithm: of three, one a multiple of 64, one of 4, one any."""
    step = rng.choice((64, 4, 1))
    return max(lo, min(hi, (_log(rng, lo, hi) + step // 2) // step * step))


def draw(rng):
    op = rng.choice(("linear", "linear", "packed", "step", "norm", "norm", "cache"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    gates = rng.choice(("channel", "preact", "tied", "tied_preact"))
    if op == "linear":
        D, T, train = _width(rng, 64, 4096), _log(rng, 1, 65536), rng.random() < 0.5
        B = max(1, min(rng.randint(1, 8), (8 * 4096 * 2048) // (T * D)))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, gates=gates, train=train)
    if op == "packed":
        D, T = _width(rng, 64, 4096), _log(rng, 64, 16384)
        return dict(op=op, N=_log(rng, 1, 96), T=T, D=D, dtype=dtype, gates=gates, train=rng.random() < 0.5)
    if op == "step":
        return dict(op=op, N=_log(rng, 1, 256), D=_width(rng, 64, 4096), dtype=dtype, gates=gates)
    if op == "norm":
        D, kind = _width(rng, 16, 8192), rng.choice(("layer", "rms"))
        rows = max(1, min(_log(rng, 1, 524288), (32768 * 2048) // D))
        return dict(op=op, rows=rows, D=D, dtype=dtype, wtype=rng.choice(("f32", dtype)), kind=kind,
                    bias=rng.random() < 0.5, gate=rng.random() < 0.5, train=rng.random() < 0.5)
    N = _log(rng, 1, 256)
    return dict(op=op, N=N, P=N + rng.randint(0, 64), H=rng.randint(1, 16), dk=rng.choice((16, 32, 64, 128)),
                dv=rng.choice((16, 32, 64, 128)), fmt=rng.choice(("e4m3", "int8")), store=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs
def _lengths(N, T, seed):
    """N lengths that add up to T, spread over a factor of about ten, one in eight of them zero."""
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(torch.randn(N, generator=g, dtype=torch.float64))
    if N > 1:
        w[torch.randperm(N, generator=g)[:N // 8]] = 0.0
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.round(torch.cumsum(w, 0) / w.sum() * T).to(torch.int32)
    return cu


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(mean, std, generator=g).to(dtype)

    st = dict(case=dict(case))
    op = case["op"]
    if op in ("linear", "packed", "step"):
        dt, D, gates = TYPES[case["dtype"]], case["D"], case["gates"]
        lead = {"linear": lambda: (case["B"], case["T"]), "packed": lambda: (case["T"],), "step": lambda: (case["N"],)}[op]()
        n = case["B"] if op == "linear" else case["N"]
        st["x"] = rand(*lead, D, dtype=dt)
        # decays of about 0.7 to 0.999 (half-lives of two to several hundred tokens), input gates over (0, 1)
        a, b = rand(*lead, D, mean=-4.0, std=1.5), None if gates.startswith("tied") else rand(*lead, D)
        if gates in ("preact", "tied_preact"):
            st["a"], st["b"] = a.to(dt), None if b is None else b.to(dt)
        else:
            st["a"], st["b"] = torch.sigmoid(-a), None if b is None else torch.sigmoid(b)
        st["h0"] = rand(n, D)
        if op == "packed":
            st["cu"] = _lengths(n, case["T"], seed).to(DEV)
        if op == "step":
            st["h_out"] = torch.empty_like(st["h0"])
        if case.get("train"):
            st["dO"], st["dh_T"] = rand(*lead, D, dtype=dt), rand(n, D)
    elif op == "norm":
        dt, wt, rows, D = TYPES[case["dtype"]], TYPES[case["wtype"]], case["rows"], case["D"]
        st["x"] = rand(rows, D, dtype=dt, mean=0.25)
        st["weight"] = rand(D, dtype=wt, mean=1.0, std=0.1)
        st["bias"] = rand(D, dtype=wt, std=0.1) if case["bias"] else None
        st["gate"] = rand(rows, D, dtype=dt) if case["gate"] else None
        if case["train"]:
            st["dy"] = rand(rows, D, dtype=dt)
    else:
        N, P, H, dk, dv = (case[k] for k in ("N", "P", "H", "dk", "dv"))
        order = torch.randperm(P, generator=torch.Generator().manual_seed(seed))
        st["slots"] = order[:N].to(torch.int32).to(DEV)
        st["cache"] = torch.zeros(P, H, dk, dv, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.zeros(P, H, dk, dtype=torch.uint8, device=DEV)
        # states whose rows differ in size, as decays of different lengths leave them
        S = rand(N, H, dk, dv) * torch.exp(rand(N, H, dk, 1))
        if case["store"]:
            st["S"] = S
        else:
            codes, e = _plain_quantise(S, case["fmt"])
            st["cache"][st["slots"].long()], st["scales"][st["slots"].long()] = codes, e
    return st


# ------------------------------------------------------------------ plain forms
def _activate(a, b, gates):
    """(a, b) in 32 bits from a gate form's tensors."""
    a = a.float()
    if gates in ("preact", "tied_preact"):
        e = torch.exp(a)
        a, na = 1.0 / (1.0 + e), 1.0 / (1.0 + 1.0 / e)
    else:
        na = 1.0 - a
    if gates.startswith("tied"):
        return a, na
    b = b.float()
    return a, 1.0 / (1.0 + torch.exp(-b)) if gates == "preact" else b


def _scan(a, u):
    """h_t = a_t h_(t-1) + u_t along axis 1 by doubling: after the step of length k every token holds 2k tokens' map."""
    a, h, k = a.clone(), u.clone(), 1
    while k < a.shape[1]:
        h[:, k:] += a[:, k:] * h[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return h


def _edges(st):
    """(first, last, alive) of the packed sequences: row indices of their first and last tokens, clamped, and whether they have any."""
    cu, T = st["cu"].long(), st["x"].shape[0]
    return cu[:-1].clamp(max=max(T - 1, 0)), (cu[1:] - 1).clamp(min=0), (cu[1:] > cu[:-1])[:, None]


def _plain_linear(st):
    case, x, h0 = st["case"], st["x"], st["h0"]
    packed, gates, dt = case["op"] == "packed", case["gates"], x.dtype
    a, b = _activate(st["a"], st["b"], gates)
    xf = x.float()
    if packed:
        first, last, alive = _edges(st)
        a, b, xf = a[None], b[None], xf[None]
        u = b * xf
        u[0].index_add_(0, first, torch.where(alive, a[0, first] * h0, 0.0))
        starts = torch.zeros(a.shape[1], device=DEV).index_add_(0, first, alive[:, 0].float())
        am = a * (starts == 0)[None, :, None]  # a sequence's first token takes nothing from the token before it
        h = _scan(am, u)
        h_T = torch.where(alive, h[0, last], h0)
    else:
        u = b * xf
        u[:, 0] += a[:, 0] * h0
        h = _scan(a, u)
        h_T = h[:, -1].clone()
    out = {"o": (h[0] if packed else h).to(dt), "h_T": h_T}
    if not case["train"]:
        return out
    # adjoints of the states, from the last token to the first: g_t = dO_t + a_(t+1) g_(t+1)
    dO = st["dO"].float()
    c = torch.zeros_like(a)
    if packed:
        dO = dO[None].clone()
        dO[0].index_add_(0, last, torch.where(alive, st["dh_T"], 0.0))
        c[:, :-1] = am[:, 1:]
    else:
        dO = dO.clone()
        dO[:, -1] += st["dh_T"]
        c[:, :-1] = a[:, 1:]
    grad = _scan(c.flip(1), dO.flip(1)).flip(1)
    hp = torch.zeros_like(h)
    hp[:, 1:] = h[:, :-1]
    if packed:
        hp *= (starts == 0)[None, :, None]
        hp[0].index_add_(0, first, torch.where(alive, h0, 0.0))
    else:
        hp[:, 0] = h0
    da, db = grad * hp, grad * xf
    if gates.startswith("tied"):
        da, db = da - db, None
    if gates in ("preact", "tied_preact"):
        e = torch.exp(st["a"].float()).reshape(a.shape)
        da = -da * a * (1.0 / (1.0 + 1.0 / e))
        db = None if db is None else db * b * (1.0 / (1.0 + torch.exp(st["b"].float()))).reshape(b.shape)
    gt = st["a"].dtype
    out["dx"] = (grad * b).to(dt)
    out["da"] = da.to(gt)
    out["db"] = None if db is None else db.to(gt)
    if packed:
        out["dh0"] = torch.where(alive, a[0, first] * grad[0, first], st["dh_T"])
        for k in ("dx", "da", "db"):
            out[k] = None if out[k] is None else out[k][0]
    else:
        out["dh0"] = a[:, 0] * grad[:, 0]
    return out


def _plain_step(st):
    a, b = _activate(st["a"], st["b"], st["case"]["gates"])
    h = a * st["h0"] + b * st["x"].float()
    st["h_out"].copy_(h)
    return {"o": h.to(st["x"].dtype), "h": st["h_out"]}


EPS = 1e-5


def _plain_norm(st):
    case, x, dt = st["case"], st["x"].float(), st["x"].dtype
    w = st["weight"].float()
    c = x - x.mean(-1, keepdim=True) if case["kind"] == "layer" else x
    r = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)
    xh = c * r
    n = xh * w
    if st["bias"] is not None:
        n = n + st["bias"].float()
    if st["gate"] is not None:
        z = st["gate"].float()
        s = 1.0 / (1.0 + torch.exp(-z))
        y = n * (z * s)
    else:
        y = n
    out = {"y": y.to(dt)}
    if not case["train"]:
        return out
    dn = st["dy"].float()
    if st["gate"] is not None:
        out["dgate"] = (dn * n * (s * (1.0 + z * (1.0 - s)))).to(dt)
        dn = dn * (z * s)
    out["dweight"] = (dn * xh).sum(0).to(st["weight"].dtype)
    if st["bias"] is not None:
        out["dbias"] = dn.sum(0).to(st["bias"].dtype)
    d = dn * w
    m = (d * xh).mean(-1, keepdim=True)
    dx = d - xh * m
    if case["kind"] == "layer":
        dx = dx - d.mean(-1, keepdim=True)
    out["dx"] = (dx * r).to(dt)
    return out


def _plain_quantise(S, fmt):
    """(codes, scales) of rows of S: values over 2^e with the smallest e that keeps the row's largest within the format's largest value."""
    top, bits = (1.75, 8) if fmt == "e4m3" else (1.984375, 6)
    m, k = torch.frexp(S.abs().amax(-1))  # amax = m 2^k, m in [0.5, 1)
    e = (k - 1 - bits + (2.0 * m > top).int()).clamp(-126, 127)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    v = torch.ldexp(S, -e[..., None])
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else torch.round(v).to(torch.int8).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _plain_cache(st):
    case, at = st["case"], st["slots"].long()
    if case["store"]:
        codes, e = _plain_quantise(st["S"], case["fmt"])
        st["cache"].index_copy_(0, at, codes)
        st["scales"].index_copy_(0, at, e)
    codes, e = st["cache"][at], st["scales"][at]
    v = codes.view(torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8).float()
    return {"S": torch.ldexp(v, e[..., None].int() - 127)}


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"linear": _plain_linear, "packed": _plain_linear, "step": _plain_step, "norm": _plain_norm,
                "cache": _plain_cache}[op](state)
    import gated_delta_rule_83_amd as g
    if op in ("linear", "packed"):
        x, a, b, h0, gates = state["x"], state["a"], state["b"], state["h0"], case["gates"]
        if not case["train"]:
            if op == "packed":
                o, h_T = g.linear_forward_varlen(x, a, b, state["cu"], h0, gates=gates)
            else:
                o, h_T = g.linear_forward(x, a, b, h0, gates=gates)
            return {"o": o, "h_T": h_T}
        names = ["x", "a", "h0"] if b is None else ["x", "a", "b", "h0"]
        leaf = {k: state[k].detach().requires_grad_() for k in names}
        if op == "packed":
            o, h_T = g.gated_linear_recurrence_varlen(leaf["x"], leaf["a"], leaf.get("b"), state["cu"], leaf["h0"], gates=gates)
        else:
            o, h_T = g.gated_linear_recurrence(leaf["x"], leaf["a"], leaf.get("b"), leaf["h0"], gates=gates)
        grads = torch.autograd.grad((o, h_T), [leaf[k] for k in names], (state["dO"], state["dh_T"]))
        return {"o": o.detach(), "h_T": h_T.detach(), "db": None, **{"d" + k: v for k, v in zip(names, grads)}}
    if op == "step":
        o = g.linear_step(state["x"], state["a"], state["b"], state["h0"], h_out=state["h_out"], gates=case["gates"])
        return {"o": o, "h": state["h_out"]}
    if op == "norm":
        fn, x, weight, bias, gate = case["kind"], state["x"], state["weight"], state["bias"], state["gate"]
        if not case["train"]:
            return {"y": g.norm_forward(x, weight, bias, gate, eps=EPS, kind=fn)}
        names = [k for k in ("x", "weight", "bias", "gate") if state[k] is not None]
        leaf = {k: state[k].detach().requires_grad_() for k in names}
        y = g.norm(leaf["x"], leaf["weight"], leaf.get("bias"), leaf.get("gate"), eps=EPS, kind=fn)
        grads = torch.autograd.grad(y, [leaf[k] for k in names], state["dy"])
        return {"y": y.detach(), **{"d" + k: v for k, v in zip(names, grads)}}
    if case["store"]:
        g.state_cache_store(state["S"], state["slots"], state["cache"], state["scales"], fmt=case["fmt"])
    return {"S": g.state_cache_load(state["cache"], state["scales"], state["slots"], fmt=case["fmt"])}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    es = {"bf16": 2, "f32": 4}
    if op in ("linear", "packed", "step"):
        e, tied = es[case["dtype"]], case["gates"].startswith("tied")
        gate = (e if case["gates"] in ("preact", "tied_preact") else 4) * (1 if tied else 2)
        rows = case["N"] if op == "step" else case["T"] * (case["B"] if op == "linear" else 1)
        n, states = rows * case["D"], (case["B"] if op == "linear" else case["N"]) * case["D"]
        bytes_, flops = n * (2 * e + gate) + states * 8, 3 * n
        if case.get("train"):  # the outputs' and last states' gradients in, the inputs' out
            bytes_, flops = bytes_ + n * (2 * e + gate) + states * 8, flops + 7 * n
        return {"bytes": bytes_, "flops": flops}
    if op == "norm":
        e, n = es[case["dtype"]], case["rows"] * case["D"]
        cols = case["D"] * es[case["wtype"]] * (2 if case["bias"] else 1)
        tensors, flops = 2 + case["gate"], 8 * n
        if case["train"]:
            tensors, flops, cols = tensors + 2 + case["gate"], flops + 14 * n, 2 * cols
        return {"bytes": n * e * tensors + cols, "flops": flops}
    rows = case["N"] * case["H"] * case["dk"]
    one = rows * (case["dv"] * 5 + 1)
    return {"bytes": 4 * case["N"] + (2 * one if case["store"] else one), "flops": rows * case["dv"] * (3 if case["store"] else 1)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_gates(st):
    a, gates = st["a"].double(), st["case"]["gates"]
    pre = gates in ("preact", "tied_preact")
    if pre:
        a = torch.sigmoid(-a)
    if gates.startswith("tied"):
        return a, torch.sigmoid(st["a"].double()) if pre else 1.0 - a
    return a, torch.sigmoid(st["b"].double()) if pre else st["b"].double()


def _exact_sequences(st, a, b, spans):
    """Token by token over `spans` (lists of (row index, first, last) of the sequences): o, h_T and every gradient."""
    train = st["case"]["train"]
    x, h0 = st["x"].double(), st["h0"].double()
    o, hT = torch.empty_like(x), h0.clone()
    gx, ga, gb, g0 = (torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), None) if train else (None,) * 4
    if train:
        g0 = st["dh_T"].double().clone()
    for n, at in spans:
        xs, as_, bs, os_ = x[at], a[at], b[at], o[at]
        xs, as_, bs = (v.unbind(-2) for v in (xs, as_, bs))
        T, h, hs = len(xs), h0[n], []
        for t in range(T):
            h = torch.addcmul(bs[t] * xs[t], as_[t], h)
            hs.append(h)
        if T:
            o[at] = torch.stack(hs, -2)
            hT[n] = h
        if train and T:
            q, dO = st["dh_T"][n].double(), st["dO"][at].double().unbind(-2)
            rx, ra, rb = [None] * T, [None] * T, [None] * T
            for t in reversed(range(T)):
                q = q + dO[t]
                rx[t], rb[t], ra[t] = bs[t] * q, xs[t] * q, (hs[t - 1] if t else h0[n]) * q
                q = as_[t] * q
            gx[at], ga[at], gb[at] = (torch.stack(v, -2) for v in (rx, ra, rb))
            g0[n] = q
    return o, hT, gx, ga, gb, g0


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "packed"):
        a, b = _exact_gates(st)
        if op == "packed":
            cu = st["cu"].tolist()
            spans = [(n, slice(cu[n], cu[n + 1])) for n in range(case["N"])]
        else:
            spans = [(slice(None), slice(None))]
        o, hT, gx, ga, gb, g0 = _exact_sequences(st, a, b, spans)
        out = {"o": o, "h_T": hT}
        if case["train"]:
            if case["gates"].startswith("tied"):
                ga, gb = ga - gb, None
            if case["gates"] in ("preact", "tied_preact"):
                ga = -ga * a * torch.sigmoid(st["a"].double())
                gb = None if gb is None else gb * b * torch.sigmoid(-st["b"].double())
            out.update(dx=gx, da=ga, db=gb, dh0=g0)
        return out
    if op == "step":
        a, b = _exact_gates(st)
        h = a * st["h0"].double() + b * st["x"].double()
        return {"o": h, "h": h}
    if op == "norm":
        names = [k for k in ("x", "weight", "bias", "gate") if st[k] is not None]
        leaf = {k: st[k].double().requires_grad_(case["train"]) for k in names}
        x = leaf["x"]
        if case["kind"] == "layer":
            y = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + EPS)
        else:
            y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        y = y * leaf["weight"]
        if "bias" in leaf:
            y = y + leaf["bias"]
        if "gate" in leaf:
            y = y * leaf["gate"] * torch.sigmoid(leaf["gate"])
        if not case["train"]:
            return {"y": y}
        grads = torch.autograd.grad(y, [leaf[k] for k in names], st["dy"].double())
        return {"y": y.detach(), **{"d" + k: v for k, v in zip(names, grads)}}
    if not case["store"]:
        codes = st["cache"][st["slots"].long()]
        if case["fmt"] == "int8":
            v = codes.double() - 256.0 * (codes > 127)
        else:  # a sign, four bits of exponent (bias 7; 0: subnormal), three of fraction
            c = codes.long()
            ex, fr = (c >> 3) & 15, (c & 7).double()
            v = torch.where(ex > 0, (1.0 + fr / 8.0) * torch.exp2(ex.double() - 7.0), fr / 8.0 * 2.0 ** -6)
            v = torch.where(c > 127, -v, v)
        return {"S": v * torch.exp2(st["scales"][st["slots"].long()].double() - 127.0)[..., None]}
    # rows over the smallest power of two that keeps them within the format, rounded to its grid, half to even
    S = st["S"].double()
    most = 448.0 if case["fmt"] == "e4m3" else 127.0
    big = S.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(big / most)))
    scale = torch.where(scale < big / most, scale * 2.0, torch.where(scale / 2.0 >= big / most, scale / 2.0, scale))
    v = S / scale
    if case["fmt"] == "int8":
        return {"S": torch.round(v) * scale}
    grid = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return {"S": torch.round(v / grid) * grid * scale}
