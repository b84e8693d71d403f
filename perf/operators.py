"""What is measured of the gated recurrence, the rotary positions and the group norm.

Each case is one pass through an operator of the package: ``prepare`` makes what a program
holds before the call, ``run`` is the call (with ``own``: the package's entry points,
without: the same mathematics in elementary torch operations), ``exact`` the definition in
64 bits.  Layouts are the package's: x, q, k [B, H, L, d], one position per row of L.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
TWO_PI = 2.0 * math.pi


# ---- cases -----------------------------------------------------------------------------
def listed():
    return [
        # one decoded token for every sequence of a small serving batch
        dict(name="recurrence-step-B8", op="recurrence_step", B=8, H=16, d=128, dtype="bf16",
             gate_dtype="bf16", gate="sigmoid", complement=True),
        # prefill / forward of a wide layer: the headline workload's shape
        dict(name="recurrence-fwd-L8192", op="recurrence_fwd", B=8, H=16, L=8192, d=128, dtype="bf16",
             gate_dtype="bf16", gate="sigmoid", complement=True, initial=False, padded=False),
        # one long document continued from a state; log gates, some rows reset (gate 0)
        dict(name="recurrence-fwd-L65536", op="recurrence_fwd", B=1, H=16, L=65536, d=64, dtype="f32",
             gate_dtype="f32", gate="log", complement=False, initial=True, padded=False),
        # training step of a layer with few heads: bf16 activations, fp32 log gates
        dict(name="recurrence-train-L16384", op="recurrence_train", B=2, H=12, L=16384, d=64, dtype="bf16",
             gate_dtype="f32", gate="log", complement=True, initial=True, padded=False),
        # a padded batch with odd sizes, one sequence empty
        dict(name="recurrence-train-padded-L777", op="recurrence_train", B=5, H=3, L=777, d=40, dtype="f32",
             gate_dtype="f32", gate="value", complement=False, initial=True, padded=True),
        # one decoded token of 64 sequences at far, unequal positions
        dict(name="rotary-step-B64", op="rotary", B=64, H=16, Hk=16, L=1, d=128, rot=128, layout="half",
             dtype="bf16", scaling="parts", far=1000000, inverse=False),
        # q and k out of one projection of a training batch
        dict(name="rotary-L8192", op="rotary", B=8, H=16, Hk=16, L=8192, d=128, rot=128, layout="half",
             dtype="bf16", scaling="none", far=0, inverse=False),
        # the gradient: rotated back into the projection's layout; part of the head, odd length
        dict(name="rotary-grad-L16383", op="rotary", B=2, H=12, Hk=12, L=16383, d=64, rot=32,
             layout="interleaved", dtype="bf16", scaling="linear", far=0, inverse=True),
        # the token mixer's output of one decoded token
        dict(name="group-norm-step-B64", op="group_norm", B=64, H=16, L=1, d=128, dtype="bf16", gated=True,
             affine=True, center=True),
        # forward behind the headline workload
        dict(name="group-norm-L8192", op="group_norm", B=8, H=16, L=8192, d=128, dtype="bf16", gated=True,
             affine=True, center=True),
        # training step behind a layer with few heads
        dict(name="group-norm-train-L16384", op="group_norm_train", B=2, H=12, L=16384, d=64, dtype="bf16",
             gated=True, affine=True, center=True),
        # odd sizes, fp32, no gate, no centring
        dict(name="group-norm-train-L333", op="group_norm_train", B=3, H=5, L=333, d=80, dtype="f32",
             gated=False, affine=True, center=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["recurrence_step", "recurrence_fwd", "recurrence_train", "rotary", "rotary",
                     "group_norm", "group_norm_train"])
    dtype = rng.choice(["bf16", "f32"])
    H = _spread(rng, 1, 24)
    d = rng.choice([64, 128, 64, 128, _spread(rng, 8, 256)])
    top = 1 << 26 if dtype == "bf16" else 1 << 25  # elements: within the largest listed case
    if op == "recurrence_step":
        return dict(op=op, B=_spread(rng, 1, 128), H=H, d=d, dtype=dtype,
                    gate_dtype=rng.choice([dtype, "f32"]), gate=rng.choice(["value", "log", "sigmoid"]),
                    complement=rng.random() < 0.5)
    L = rng.choice([1, _spread(rng, 2, 2000), _spread(rng, 2, 65536), _spread(rng, 1024, 65536)])
    L = min(L, top // (H * d))
    B = _spread(rng, 1, max(1, min(64, top // (H * d * L))))
    if op.startswith("recurrence"):
        return dict(op=op, B=B, H=H, L=L, d=d, dtype=dtype, gate_dtype=rng.choice([dtype, "f32"]),
                    gate=rng.choice(["value", "log", "sigmoid"]), complement=rng.random() < 0.5,
                    initial=rng.random() < 0.5, padded=rng.random() < 0.3)
    if op == "rotary":
        d += d % 2
        return dict(op=op, B=B, H=H, Hk=rng.choice([h for h in range(1, H + 1) if H % h == 0]), L=L, d=d,
                    rot=rng.choice([d, d // 4 * 2 or 2]), layout=rng.choice(["half", "interleaved"]),
                    dtype=dtype, scaling=rng.choice(["none", "linear", "parts"]),
                    far=rng.choice([0, 100000, 1000000]), inverse=rng.random() < 0.3)
    return dict(op=op, B=B, H=H, L=L, d=d, dtype=dtype, gated=rng.random() < 0.6,
                affine=rng.random() < 0.7, center=rng.random() < 0.7)


# ---- inputs ----------------------------------------------------------------------------
ROTARY_BASE, ROTARY_FACTOR, ROTARY_ORIGINAL = 10000.0, 8.0, 8192


def _gate_input(case, shape, gen):
    """Gate inputs as a layer gives them: mostly long memory, some quick; one row in a
    thousand forgets everything (a document's first row)."""
    n = torch.randn(shape, generator=gen, device="cuda")
    reset = torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") < 1e-3
    if case["gate"] == "sigmoid":
        return n.mul_(1.5).add_(2.5)
    if case["gate"] == "log":
        n = -torch.nn.functional.softplus(n.mul_(1.5).sub_(2.5))
        return n.masked_fill_(reset, float("-inf"))
    return torch.sigmoid_(n.mul_(1.5).add_(2.5)).masked_fill_(reset, 0.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape, dtype=t):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    B, H, d, L = case["B"], case["H"], case["d"], case.get("L", 1)
    s = dict(case)
    if op.startswith("recurrence"):
        g = TYPES[case["gate_dtype"]]
        shape = (B, H, d) if op == "recurrence_step" else (B, H, L, d)
        s["x"] = normal(*shape)
        s["g"] = _gate_input(case, shape, gen).to(g)
        if op == "recurrence_step":
            s["state"] = normal(B, H, d, dtype=torch.float32)
            return s
        s["h0"] = normal(B, H, d, dtype=torch.float32) if case["initial"] else None
        s["lengths"] = None
        if case["padded"]:
            n = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            n[0] = L
            if B > 1:
                n[1] = 0
            s["lengths"] = n
        if op == "recurrence_train":
            s["dout"] = normal(*shape)
            s["dlast"] = normal(B, H, d, dtype=torch.float32)
        return s
    if op == "rotary":
        Hk = case["Hk"]
        if case["inverse"]:
            s["q"], s["k"] = normal(B, H, L, d), normal(B, Hk, L, d)
        else:  # one projection's output [B, L, (H + Hk + Hk) d]: q, k are views of it
            rows = normal(B, L, H + 2 * Hk, d)
            s["q"] = rows[:, :, :H].transpose(1, 2)
            s["k"] = rows[:, :, H:H + Hk].transpose(1, 2)
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["positions"] = start + torch.arange(L, device="cuda", dtype=torch.int32)
        if own:
            import chunkwise_causal_linear_gb300 as la
            s["table"] = la.rotary_table(case["rot"], base=ROTARY_BASE, scaling=case["scaling"],
                                         factor=ROTARY_FACTOR, original_length=ROTARY_ORIGINAL)
        else:
            s["theta"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        return s
    s["x"] = normal(B, H, L, d)
    s["gate"] = normal(B, L, H * d) if case["gated"] else None
    s["w"] = 1 + 0.1 * normal(H * d, dtype=torch.float32) if case["affine"] else None
    s["b"] = 0.1 * normal(H * d, dtype=torch.float32) if case["affine"] else None
    if op == "group_norm_train":
        s["dout"] = normal(B, L, H * d)
    return s


def _frequencies(case):
    """theta_j = base^(-2j/rot), scaled for contexts longer than the original: all divided by
    the factor (linear), or those of few turns over the original length only (parts: none
    above 32 turns, all below 1, in between mixed)."""
    out = []
    for j in range(case["rot"] // 2):
        theta = ROTARY_BASE ** (-2.0 * j / case["rot"])
        if case["scaling"] == "linear":
            theta /= ROTARY_FACTOR
        elif case["scaling"] == "parts":
            keep = min(1.0, max(0.0, (ROTARY_ORIGINAL * theta / TWO_PI - 1.0) / (32.0 - 1.0)))
            theta = theta * keep + theta / ROTARY_FACTOR * (1.0 - keep)
        out.append(theta)
    return out


# ---- one pass --------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import chunkwise_causal_linear_gb300 as la
    op = s["op"]
    if op == "recurrence_step":
        out = la.recurrence_step(s["x"], s["g"], s["state"], gate_kind=s["gate"], complement=s["complement"])
        return {"out": out, "state": s["state"]}
    if op.startswith("recurrence"):
        kw = dict(gate_kind=s["gate"], complement=s["complement"], lengths=s["lengths"])
        if op == "recurrence_fwd":
            out, last = la.recurrence_fwd(s["x"], s["g"], h0=s["h0"], **kw)
            return {"out": out, "last": last}
        out, last, chunks = la.recurrence_fwd(s["x"], s["g"], h0=s["h0"], save_chunks=True, **kw)
        dx, dg, dh0 = la.recurrence_bwd(s["x"], s["g"], chunks, s["dout"], dh_last=s["dlast"], **kw)
        return {"out": out, "last": last, "dx": dx, "dg": dg, "dh0": dh0}
    if op == "rotary":
        if not s["inverse"]:
            q, k = la.rotary(s["q"], s["k"], s["table"], positions=s["positions"], layout=s["layout"])
            return {"q": q, "k": k}
        rows, q, k = _projection_views(s)
        la.rotary(s["q"], s["k"], s["table"], positions=s["positions"], layout=s["layout"], inverse=True,
                  q_out=q, k_out=k)
        return {"rows": rows}
    kw = dict(gate=s["gate"], center=s["center"])
    out = la.group_norm_fwd(s["x"], s["w"], s["b"], **kw)
    if op == "group_norm":
        return {"out": out}
    dx, dgate, dw, db = la.group_norm_bwd(s["x"], s["dout"], s["w"], s["b"], **kw)
    return _present(out=out, dx=dx, dgate=dgate, dw=dw, db=db)


def _projection_views(s):
    B, H, L, d = s["q"].shape
    Hk = s["k"].shape[1]
    rows = torch.empty((B, L, H + Hk, d), dtype=s["q"].dtype, device=s["q"].device)
    return rows, rows[:, :, :H].transpose(1, 2), rows[:, :, H:].transpose(1, 2)


def _present(**outs):
    return {k: v for k, v in outs.items() if v is not None}


# ---- the plain form --------------------------------------------------------------------
def _gates(kind, g):
    """(a, 1 - a, da/dg) in the gate's own precision, 1 - a without cancellation."""
    if kind == "value":
        return g, 1 - g, torch.ones_like(g)
    if kind == "log":
        a = torch.exp(g)
        return a, -torch.expm1(g), a
    a, c = torch.sigmoid(g), torch.sigmoid(-g)
    return a, c, a * c


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 2, by doubling: after the step of width n, row t
    holds the product of the gates and the sum of the inputs of rows t-2n+1 .. t."""
    a, b = a.clone(), b.clone()
    n, L = 1, a.shape[2]
    while n < L:
        b[:, :, n:] = torch.addcmul(b[:, :, n:], a[:, :, n:], b[:, :, :-n])
        a[:, :, n:] = a[:, :, n:] * a[:, :, :-n]
        n *= 2
    return b


def _run_plain(s):
    op, t = s["op"], TYPES[s["dtype"]]
    if op == "recurrence_step":
        a, c, _ = _gates(s["gate"], s["g"].float())
        s["state"].copy_(a * s["state"] + (c if s["complement"] else 1.0) * s["x"].float())
        return {"out": s["state"].to(t), "state": s["state"]}
    if op.startswith("recurrence"):
        return _recurrence_plain(s, op == "recurrence_train")
    if op == "rotary":
        return _rotary_plain(s)
    return _group_norm_plain(s, op == "group_norm_train")


def _recurrence_plain(s, train):
    t, gt = TYPES[s["dtype"]], TYPES[s["gate_dtype"]]
    x, (a, c, slope) = s["x"].float(), _gates(s["gate"], s["g"].float())
    L, keep = x.shape[2], None
    if s["lengths"] is not None:  # rows behind a sequence's end keep the state
        keep = (torch.arange(L, device=x.device) < s["lengths"][:, None])[:, None, :, None]
        a = torch.where(keep, a, 1.0)
    b = x * c if s["complement"] else x.clone()
    if keep is not None:
        b = torch.where(keep, b, 0.0)
    if s["h0"] is not None:
        b[:, :, 0] += a[:, :, 0] * s["h0"]
    h = _scan(a, b)
    last = h[:, :, -1].clone()
    out = (h if keep is None else torch.where(keep, h, 0.0)).to(t)
    if not train:
        return {"out": out, "last": last}
    e = s["dout"].float()
    if keep is not None:
        e = torch.where(keep, e, 0.0)
    else:
        e = e.clone()
    e[:, :, -1] += s["dlast"]
    later = torch.ones_like(a)
    later[:, :, :-1] = a[:, :, 1:]
    e = _scan(later.flip(2), e.flip(2)).flip(2)
    before = torch.zeros_like(h)
    before[:, :, 1:] = h[:, :, :-1]
    if s["h0"] is not None:
        before[:, :, 0] = s["h0"]
    dh0 = a[:, :, 0] * e[:, :, 0]
    dx = e * c if s["complement"] else e
    dg = e * (before - x if s["complement"] else before) * slope
    if keep is not None:
        dx, dg = torch.where(keep, dx, 0.0), torch.where(keep, dg, 0.0)
    return {"out": out, "last": last, "dx": dx.to(t), "dg": dg.to(gt), "dh0": dh0}


def _rotary_plain(s):
    angle = s["positions"].double()[:, None, :, None] * s["theta"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if s["inverse"]:
        sin = -sin
    half, rot = s["layout"] == "half", s["rot"]

    def turn(x):
        y, z = x.clone(), x[..., :rot].float()
        u, v = (z[..., :rot // 2], z[..., rot // 2:]) if half else (z[..., 0::2], z[..., 1::2])
        p, r = u * cos - v * sin, u * sin + v * cos
        y[..., :rot] = (torch.cat((p, r), -1) if half else torch.stack((p, r), -1).flatten(-2)).to(y.dtype)
        return y

    q, k = turn(s["q"]), turn(s["k"])
    if not s["inverse"]:
        return {"q": q, "k": k}
    rows, qv, kv = _projection_views(s)
    qv.copy_(q)
    kv.copy_(k)
    return {"rows": rows}


GROUP_NORM_EPS = 1e-5


def _rows(x):
    """[B, H, L, d] -> [B, L, H, d]"""
    return x.transpose(1, 2)


def _group_norm_plain(s, train):
    t = TYPES[s["dtype"]]
    x = _rows(s["x"]).float()
    B, L, H, d = x.shape
    w = s["w"].view(H, d) if s["w"] is not None else 1.0
    xc = x - x.mean(-1, keepdim=True) if s["center"] else x
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + GROUP_NORM_EPS)
    xh = xc * rstd
    y = xh * w + (s["b"].view(H, d) if s["b"] is not None else 0.0)
    z = s["gate"].float().view(B, L, H, d) if s["gate"] is not None else y
    sig = torch.sigmoid(z)
    act = z * sig
    out = (y * act if s["gate"] is not None else act).reshape(B, L, H * d).to(t)
    if not train:
        return {"out": out}
    do = s["dout"].float().view(B, L, H, d)
    slope = sig * (1 + z * (1 - sig))
    if s["gate"] is not None:
        dy, dgate = do * act, (do * y * slope).reshape(B, L, H * d).to(t)
    else:
        dy, dgate = do * slope, None
    dw = (dy * xh).sum((0, 1)).view(-1) if s["w"] is not None else None
    db = dy.sum((0, 1)).view(-1) if s["b"] is not None else None
    dxh = dy * w
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if s["center"]:
        dx = dx - dxh.mean(-1, keepdim=True)
    return _present(out=out, dx=_rows(dx * rstd).contiguous().to(t), dgate=dgate, dw=dw, db=db)


# ---- the definition in 64 bits -----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        theta = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        angle = s["positions"].double()[:, None, :, None] * theta
        unit = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)

        def turn(x):
            rot = case["rot"]
            z = x[..., :rot].double()
            pairs = (z.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half"
                     else z.unflatten(-1, (rot // 2, 2)))
            r = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
            r = r.transpose(-1, -2) if case["layout"] == "half" else r
            return torch.cat((r.flatten(-2), x[..., rot:].double()), -1)

        q, k = turn(s["q"]), turn(s["k"])
        return {"rows": torch.cat((q, k), 1).transpose(1, 2)} if case["inverse"] else {"q": q, "k": k}
    if op.startswith("group_norm"):
        return _group_norm_exact(s, op == "group_norm_train")
    return _recurrence_exact(s)


def _recurrence_exact(s):
    """The recurrence row by row, forwards and (for the gradients) backwards."""
    step = s["op"] == "recurrence_step"
    x, g = s["x"].double(), s["g"].double()
    if step:
        x, g, h = x[:, :, None], g[:, :, None], s["state"].double()
    else:
        h = torch.zeros_like(x[:, :, 0]) if s["h0"] is None else s["h0"].double()
    L = x.shape[2]
    if s["gate"] == "value":
        a = g
    else:
        a = torch.exp(g) if s["gate"] == "log" else 1 / (1 + torch.exp(-g))
    # 1 - a, for the log gate by expm1; the sigmoid's is small only to a 64-bit rounding
    w = (-torch.expm1(g) if s["gate"] == "log" else 1 - a) if s["complement"] else torch.ones_like(a)
    live = None
    if not step and s["lengths"] is not None:
        live = torch.arange(L, device=x.device) < s["lengths"][:, None]
    train = s["op"] == "recurrence_train"
    out, before = torch.zeros_like(x), torch.zeros_like(x) if train else None
    for i in range(L):
        if train:
            before[:, :, i] = h
        new = torch.addcmul(w[:, :, i] * x[:, :, i], a[:, :, i], h)
        if live is not None:
            on = live[:, i, None, None]
            h = torch.where(on, new, h)
            out[:, :, i] = torch.where(on, h, 0.0)
        else:
            h = new
            out[:, :, i] = h
    if step:
        return {"out": h, "state": h}
    if not train:
        return {"out": out, "last": h}
    carry, dout = s["dlast"].double(), s["dout"].double()  # carry: a_{t+1} e_{t+1}
    e = torch.zeros_like(x)
    for i in reversed(range(L)):
        now = dout[:, :, i] + carry
        if live is not None:
            on = live[:, i, None, None]
            now = torch.where(on, now, 0.0)
            carry = torch.where(on, a[:, :, i] * now, carry)
        else:
            carry = a[:, :, i] * now
        e[:, :, i] = now
    slope = {"value": torch.ones_like(a), "log": a, "sigmoid": a * (1 - a)}[s["gate"]]
    dg = e * slope * (before - x if s["complement"] else before)
    return {"out": out, "last": h, "dx": e * w, "dg": dg, "dh0": carry}


def _group_norm_exact(s, train):
    """Forward from the definition, gradients by differentiating it."""
    x = s["x"].double().requires_grad_(train)
    B, H, L, d = x.shape
    leaves = {"dx": x}
    y = x.permute(0, 2, 1, 3)
    if s["center"]:
        y = y - y.sum(-1, keepdim=True) / d
    y = (y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + GROUP_NORM_EPS)).reshape(B, L, H * d)
    if s["gate"] is not None:
        leaves["dgate"] = s["gate"].double().requires_grad_(train)
    if s["w"] is not None:
        leaves["dw"], leaves["db"] = s["w"].double().requires_grad_(train), s["b"].double().requires_grad_(train)
        y = y * leaves["dw"] + leaves["db"]
    out = y * leaves["dgate"] / (1 + torch.exp(-leaves["dgate"])) if s["gate"] is not None else y / (1 + torch.exp(-y))
    if not train:
        return {"out": out}
    grads = dict(zip(leaves, torch.autograd.grad(out, list(leaves.values()), s["dout"].double())))
    return {"out": out.detach(), **{k: grads[k] for k in ("dx", "dgate", "dw", "db") if k in grads}}


# ---- what a pass cannot do without --------------------------------------------------------
def work(case):
    """Each input read once, each output written once; the operations of the formulas."""
    op, z = case["op"], BYTES[case["dtype"]]
    rows, d = case["B"] * case["H"], case["d"]
    E = rows * case.get("L", 1) * d
    if op.startswith("recurrence"):
        zg, state = BYTES[case["gate_dtype"]], 4 * rows * d
        if op == "recurrence_step":
            return {"bytes": E * (2 * z + zg) + 2 * state, "flops": 6 * E}
        n = E * (2 * z + zg) + state * (2 if case["initial"] else 1)
        if op == "recurrence_fwd":
            return {"bytes": n, "flops": 6 * E}
        return {"bytes": n + E * (2 * z + zg) + 2 * state, "flops": 20 * E}
    if op == "rotary":
        E = case["B"] * (case["H"] + case["Hk"]) * case["L"] * d
        return {"bytes": 2 * E * z + 4 * case["B"] * case["L"], "flops": 3 * E * case["rot"] // d}
    arrays = 3 if case["gated"] else 2
    n = E * z * arrays + (8 * case["H"] * d if case["affine"] else 0)
    if op == "group_norm":
        return {"bytes": n, "flops": 12 * E}
    n += E * z * arrays + (8 * case["H"] * d if case["affine"] else 0)
    return {"bytes": n, "flops": 40 * E}
