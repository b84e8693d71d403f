"""What is measured of the gated attention and the norms around a block.

Each case is one pass through an operator of the package: ``prepare`` makes what a program
holds before the call, ``run`` is the call (with ``own``: the package's entry points,
without: the same mathematics in elementary torch operations), ``exact`` the definition in
64 bits.

Gated attention, for every head (rows t, a state S of dk x dv, a decay a_t = exp(g_t)):

    S_t = a_t S_{t-1} + k_t v_t^T,      out_t = scale q_t^T S_t,

with q [B, H, L, dk], k [B, Hk, L, dk], v [B, Hk, L, dv] (H / Hk heads share a key head),
g a constant of each head ([H]) or one per token and head ([B, H, L]), -inf forgetting all
before its row.  The norms around a block (rows of d channels):

    h = residual_scale r + branch_scale act(gate) (norm(y) w_post + b_post),
    n = norm(h) w_pre + b_pre.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ---- cases -----------------------------------------------------------------------------
def listed():
    return [
        # one decoded token of a small serving batch, retention's constant decays
        dict(name="gated-step-B8", op="gated_step", B=8, H=16, Hk=16, dk=128, dv=128, dtype="bf16",
             gates="head", slots=False),
        # one decoded token of 64 requests whose states lie in a pool; shared key heads
        dict(name="gated-step-B64-slots", op="gated_step", B=64, H=32, Hk=8, dk=128, dv=128, dtype="bf16",
             gates="token", slots=True),
        # the prompts of a full batch, the headline workload's shape, gates from the tokens
        dict(name="gated-prompt-L8192", op="gated_fwd", B=8, H=16, Hk=16, L=8192, dk=128, dv=128, dtype="bf16",
             gates="token", initial=False, padded=False, slots=False),
        # one long prompt continued from its state in the pool, shared key heads
        dict(name="gated-prompt-L65536", op="gated_fwd", B=1, H=16, Hk=4, L=65536, dk=64, dv=64, dtype="bf16",
             gates="head", initial=True, padded=False, slots=True),
        # a few padded prompts of odd sizes in fp32, one of them empty
        dict(name="gated-prompt-padded-L777", op="gated_fwd", B=5, H=6, Hk=3, L=777, dk=40, dv=24, dtype="f32",
             gates="token", initial=True, padded=True, slots=False),
        # training step of a layer with few heads
        dict(name="gated-train-L16384", op="gated_train", B=2, H=12, Hk=12, L=16384, dk=64, dv=64, dtype="bf16",
             gates="token", initial=False, padded=False),
        # training step with documents packed into rows (resets), two heads to a key head
        dict(name="gated-train-L2047", op="gated_train", B=4, H=8, Hk=4, L=2047, dk=128, dv=128, dtype="bf16",
             gates="token", initial=True, padded=True),
        # small fp32 training step, odd sizes
        dict(name="gated-train-L333", op="gated_train", B=3, H=5, Hk=1, L=333, dk=80, dv=64, dtype="f32",
             gates="head", initial=True, padded=False),
        # the norms around a layer for one decoded token of 64 requests
        dict(name="block-norm-step-B64", op="block_norm", B=64, L=1, d=2048, dtype="bf16", residual="f32",
             post="rms", pre="rms", gated=True, affine=True),
        # forward of the headline workload's layer (16 heads of 128 channels)
        dict(name="block-norm-L8192", op="block_norm", B=8, L=8192, d=2048, dtype="bf16", residual="bf16",
             post="rms", pre="rms", gated=True, affine=True),
        # training step of the layer with 12 heads of 64 channels, fp32 residual stream
        dict(name="block-norm-train-L16384", op="block_norm_train", B=2, L=16384, d=768, dtype="bf16",
             residual="f32", post="rms", pre="layer", gated=True, affine=True),
        # odd sizes, fp32, a layer scale in the place of the norm behind the block
        dict(name="block-norm-train-L333", op="block_norm_train", B=3, L=333, d=400, dtype="f32",
             residual="f32", post="none", pre="layer", gated=False, affine=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gated_step", "gated_fwd", "gated_fwd", "gated_train", "block_norm", "block_norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("block_norm"):
        d = rng.choice([768, 2048, _spread(rng, 16, 8192), 8 * _spread(rng, 2, 1024)])
        rows = max(1, min(1 << 16, ((1 << 27) if op == "block_norm" and dtype == "bf16" else (1 << 24)) // d))
        L = rng.choice([1, _spread(rng, 1, rows), _spread(rng, max(1, rows // 64), rows)])
        return dict(op=op, B=_spread(rng, 1, max(1, min(64, rows // L))), L=L, d=d, dtype=dtype,
                    residual=rng.choice([dtype, "f32"]), post=rng.choice(["none", "rms", "rms", "layer"]),
                    pre=rng.choice(["rms", "layer"]), gated=rng.random() < 0.6, affine=rng.random() < 0.8)
    Hk = _spread(rng, 1, 16)
    H = Hk * rng.choice([1, 1, 2, 4])
    dk = rng.choice([64, 128, 64, 128, _spread(rng, 8, 256)])
    dv = rng.choice([dk, dk, dk, 64, _spread(rng, 8, 256)])
    gates = rng.choice(["head", "token"])
    if op == "gated_step":
        return dict(op=op, B=_spread(rng, 1, 64), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, gates=gates,
                    slots=rng.random() < 0.5)
    # rows of all heads: the largest listed case's work, less in fp32 and for odd sizes
    top = (1 << 27) // (128 * max(1, max(dk, dv) // 64))
    top //= 1 if dtype == "bf16" and op == "gated_fwd" else 4
    L = rng.choice([1, _spread(rng, 2, 600), _spread(rng, 64, 16384), _spread(rng, 1024, 65536)])
    L = max(1, min(L, top // H))
    B = _spread(rng, 1, max(1, min(32, top // (H * L))))
    case = dict(op=op, B=B, H=H, Hk=Hk, L=L, dk=dk, dv=dv, dtype=dtype, gates=gates,
                initial=rng.random() < 0.5, padded=rng.random() < 0.4)
    if op == "gated_fwd":
        case["slots"] = rng.random() < 0.4
    return case


# ---- inputs ------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, op, B = TYPES[case["dtype"]], case["op"], case["B"]

    def normal(*shape, dtype=t):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    s = dict(case)
    if op.startswith("block_norm"):
        L, d, f32 = case["L"], case["d"], torch.float32
        s["y"], s["r"] = normal(B, L, d), (2 * normal(B, L, d, dtype=f32)).to(TYPES[case["residual"]])
        s["gate"] = normal(B, L, d) if case["gated"] else None
        for name, one in (("post_w", 1.0), ("post_b", 0.0), ("pre_w", 1.0), ("pre_b", 0.0)):
            centred = case["post" if name.startswith("post") else "pre"] == "layer"
            has = case["affine"] and (name.endswith("w") or centred)
            s[name] = one + 0.1 * normal(d, dtype=f32) if has else None
        s["residual_scale"], s["branch_scale"] = 1.0, 0.5
        if op == "block_norm_train":
            s["dh"], s["dn"] = normal(B, L, d, dtype=TYPES[case["residual"]]), normal(B, L, d)
        return s
    H, Hk, dk, dv, L = case["H"], case["Hk"], case["dk"], case["dv"], case.get("L", 1)
    s["scale"] = dk ** -0.5
    # one projection's output [B, L, heads, channels]: q, k, v are views of it
    rows = normal(B, L, H * dk + Hk * (dk + dv))
    q, k, v = rows.split([H * dk, Hk * dk, Hk * dv], -1)
    s["q"], s["k"], s["v"] = (x.unflatten(-1, (n, -1)).transpose(1, 2) for x, n in ((q, H), (k, Hk), (v, Hk)))
    if op == "gated_step":
        s["q"], s["k"], s["v"] = (s[n][:, :, 0] for n in "qkv")
    if case["gates"] == "head":  # retention: 1 - 2^-5, 1 - 2^-6, ... over the heads
        s["g"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.arange(H, device="cuda") / max(1, H - 1))).float()
    else:  # mostly long memory, some quick; one row in five hundred begins a document
        shape = (B, H) if op == "gated_step" else (B, H, L)
        g = -torch.nn.functional.softplus(torch.randn(shape, generator=gen, device="cuda").mul_(1.5).sub_(3.0))
        first = torch.rand((B, 1) + shape[2:], generator=gen, device="cuda") < 0.002
        s["g"] = g.masked_fill_(first, float("-inf"))
    s["lengths"] = s["slots"] = s["state0"] = None
    n = B
    if case.get("slots"):
        n = B + B // 4 + 1
        s["slots"] = torch.randperm(n, generator=gen, device="cuda")[:B].to(torch.int32)
    if op == "gated_step" or case.get("initial") or case.get("slots"):
        s["state0"] = normal(n, H, dk, dv, dtype=torch.float32)
    if case.get("padded"):
        lengths = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        lengths[0] = L
        if B > 1:
            lengths[1] = 0
        s["lengths"] = lengths
    if op == "gated_train":
        s["dout"] = normal(B, L, H, dv).transpose(1, 2)
        s["dstate"] = normal(B, H, dk, dv, dtype=torch.float32)
    return s


# ---- one pass ------------------------------------------------------------------------------
def _present(**outs):
    return {k: v for k, v in outs.items() if v is not None}


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import chunkwise_causal_linear_gb300 as la
    op = s["op"]
    if op == "gated_step":
        out = la.gated_step(s["q"], s["k"], s["v"], s["g"], s["state0"], scale=s["scale"], slots=s["slots"])
        return {"out": out, "state": s["state0"]}
    if op.startswith("gated"):
        out, last = la.gated_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], state0=s["state0"],
                                 lengths=s["lengths"], slots=s["slots"],
                                 state=s["state0"] if s["slots"] is not None else None)
        if op == "gated_fwd":
            return {"out": out, "state": last}
        dq, dk, dv, dg, ds = la.gated_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], scale=s["scale"],
                                          state0=s["state0"], lengths=s["lengths"], dstate=s["dstate"])
        return _present(out=out, state=last, dq=dq, dk=dk, dv=dv, dg=dg,
                        dstate0=ds if s["state0"] is not None else None)
    kw = {k: s[k] for k in ("post", "pre", "gate", "post_w", "post_b", "pre_w", "pre_b", "residual_scale",
                            "branch_scale")}
    args = dict(gate=kw["gate"], activation="silu", post_norm=kw["post"], post_weight=kw["post_w"],
                post_bias=kw["post_b"], pre_norm=kw["pre"], pre_weight=kw["pre_w"], pre_bias=kw["pre_b"],
                residual_scale=kw["residual_scale"], branch_scale=kw["branch_scale"], eps=EPS)
    h, n = la.block_norm_fwd(s["y"], s["r"], **args)
    if op == "block_norm":
        return {"h": h, "n": n}
    return _present(h=h, n=n, **la.block_norm_bwd(s["y"], s["r"], s["dh"], s["dn"], **args))


# ---- the plain form --------------------------------------------------------------------
CHUNK = 64  # rows whose pairs are formed; longer chunks form more pairs, shorter ones more states


def _run_plain(s):
    op = s["op"]
    if op == "gated_step":
        return _step_plain(s)
    if op.startswith("gated"):
        return _gated_plain(s, op == "gated_train")
    return _block_norm_plain(s, op == "block_norm_train")


def _step_plain(s):
    g, n = s["g"], s["q"].shape[1] // s["k"].shape[1]
    a = torch.exp(g).expand(s["q"].shape[:2])[..., None, None]
    k, v = (s[x].float().repeat_interleave(n, 1) for x in "kv")
    state = s["state0"] if s["slots"] is None else s["state0"][s["slots"].long()]
    state = a * state + k[..., None] * v[..., None, :]
    out = s["scale"] * (s["q"].float()[..., None] * state).sum(2)
    if s["slots"] is None:
        s["state0"].copy_(state)
    else:
        s["state0"][s["slots"].long()] = state
    return {"out": out.to(s["q"].dtype), "state": s["state0"]}


def _cut(x, L):
    """[B, H, L, ...] -> [B, H, chunks, CHUNK, ...], zeros behind the last row."""
    n = -(-L // CHUNK)
    pad = x.new_zeros(x.shape[:2] + (n * CHUNK - L,) + x.shape[3:])
    return torch.cat((x, pad), 2).unflatten(2, (n, CHUNK))


def _scan(a, b):
    """S_c = a_c S_{c-1} + b_c along dim 2, by doubling (a: a number per chunk)."""
    a, n, N = a.clone(), 1, a.shape[2]
    while n < N:
        b[:, :, n:] = torch.addcmul(b[:, :, n:], a[:, :, n:, None, None], b[:, :, :-n])
        a[:, :, n:] = a[:, :, n:] * a[:, :, :-n]
        n *= 2
    return b


def _weights(g):
    """Decays of the chunks [..., CHUNK] of log decays, through 64-bit sums: (from row j to row i >= j,
    from the chunk's start to row i, from row j to its end, over all of it), 0 across a row of -inf."""
    reset = torch.isneginf(g)
    G, part = g.masked_fill(reset, 0.0).double().cumsum(-1), reset.cumsum(-1)
    w = torch.exp((G[..., :, None] - G[..., None, :]).clamp_(max=0.0).float())
    w = w.masked_fill_(part[..., :, None] != part[..., None, :], 0.0).tril_()
    start = torch.exp(G).masked_fill(part != 0, 0.0).float()
    end = torch.exp(G[..., -1:] - G).masked_fill(part != part[..., -1:], 0.0).float()
    return w, start, end, start[..., -1]


def _shared(x, Hk):
    """Sum over the heads of each key head."""
    return x.unflatten(1, (Hk, -1)).sum(2)


def _gated_plain(s, train):
    t, L, H, Hk = s["q"].dtype, s["q"].shape[2], s["q"].shape[1], s["k"].shape[1]
    B = s["q"].shape[0]
    q = _cut(s["q"].float(), L)
    k, v = (_cut(s[x].float().repeat_interleave(H // Hk, 1), L) for x in "kv")
    g = s["g"] if s["g"].dim() == 3 else s["g"][None, :, None].expand(B, H, L)
    keep = None
    if s["lengths"] is not None:
        keep = (torch.arange(L, device=q.device) < s["lengths"][:, None])[:, None, :, None]
        g = torch.where(keep[..., 0], g, 0.0)
        k = torch.where(_cut(keep, L), k, 0.0)
    w, start, end, whole = _weights(_cut(g, L))
    scores = q @ k.transpose(-1, -2)
    add = (k * end[..., None]).transpose(-1, -2) @ v
    first = s["state0"] if s["slots"] is None or s["state0"] is None else s["state0"][s["slots"].long()]
    if first is not None:
        add[:, :, 0] += whole[:, :, 0, None, None] * first
    after = _scan(whole, add)
    before = torch.zeros_like(after)
    before[:, :, 1:] = after[:, :, :-1]
    if first is not None:
        before[:, :, 0] = first
    out = s["scale"] * ((w * scores) @ v + start[..., None] * (q @ before))

    def rows(x, to=t):
        x = x.flatten(2, 3)[:, :, :L]
        return (x if keep is None else torch.where(keep, x, 0.0)).to(to)

    last = after[:, :, -1].clone()
    if s["slots"] is not None:
        s["state0"][s["slots"].long()] = last
        last = s["state0"]
    outs = {"out": rows(out), "state": last}
    if not train:
        return outs
    do = s["dout"].float() * s["scale"]
    do = _cut(do if keep is None else torch.where(keep, do, 0.0), L)
    # the gradient of the state behind each chunk, from the last one on
    give = (q * start[..., None]).transpose(-1, -2) @ do
    later = torch.zeros_like(give)
    later[:, :, :-1] = give[:, :, 1:]
    later[:, :, -1] = s["dstate"]
    decay = torch.ones_like(whole)
    decay[:, :, :-1] = whole[:, :, 1:]
    decay[:, :, -1] = 0.0
    after_d = _scan(decay.flip(2), later.flip(2)).flip(2)
    if s["state0"] is not None:
        outs["dstate0"] = whole[:, :, 0, None, None] * after_d[:, :, 0] + give[:, :, 0]
    pairs = w * (do @ v.transpose(-1, -2))
    old = start[..., None] * (do @ before.transpose(-1, -2))
    new = end[..., None] * (v @ after_d.transpose(-1, -2))
    outs["dq"] = rows(pairs @ k + old)
    dk = pairs.transpose(-1, -2) @ q + new
    dv = (w * scores).transpose(-1, -2) @ do + end[..., None] * (k @ after_d)
    if keep is not None:
        dk, dv = (torch.where(_cut(keep, L), x, 0.0) for x in (dk, dv))
    outs["dk"], outs["dv"] = ((_shared(x, Hk).flatten(2, 3)[:, :, :L]).to(t) for x in (dk, dv))
    # log decay of row t: every pair (earlier row or state, later row or state) across it
    W = (pairs * scores).tril_(-1)
    W = W.flip(-2).cumsum(-2).flip(-2).cumsum(-1)
    dg = torch.zeros_like(start)
    dg[..., 1:] = W.diagonal(-1, -2, -1)
    dg += (old * q).sum(-1).flip(-1).cumsum(-1).flip(-1)
    into = (new * k).sum(-1)
    dg += into.cumsum(-1) - into
    dg += (whole * (after_d * before).sum((-1, -2)))[..., None]
    dg = rows(dg[..., None], torch.float32)[..., 0]
    outs["dg"] = dg if s["g"].dim() == 3 else dg.sum((0, 2))
    return outs


def _normed(x, kind):
    """(xh, 1/deviation) of rows."""
    xc = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    return xc * rstd, rstd


def _normed_back(dxh, xh, rstd, kind):
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - dxh.mean(-1, keepdim=True)
    return dx * rstd


def _block_norm_plain(s, train):
    t, rt = s["y"].dtype, s["r"].dtype
    y, w1, w2 = s["y"].float(), s["post_w"], s["pre_w"]
    yh, yr = _normed(y, s["post"]) if s["post"] != "none" else (y, None)
    u = yh * w1 if w1 is not None else yh
    u = u + s["post_b"] if s["post_b"] is not None else u
    act = 1.0
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = torch.sigmoid(z)
        act = z * sig
    h = s["residual_scale"] * s["r"].float() + s["branch_scale"] * act * u
    hh, hr = _normed(h, s["pre"])
    n = hh * w2 if w2 is not None else hh
    n = n + s["pre_b"] if s["pre_b"] is not None else n
    outs = {"h": h.to(rt), "n": n.to(t)}
    if not train:
        return outs
    dn = s["dn"].float()
    dH = s["dh"].float() + _normed_back(dn * w2 if w2 is not None else dn, hh, hr, s["pre"])
    outs["dr"] = (s["residual_scale"] * dH).to(rt)
    db = s["branch_scale"] * dH
    if s["gate"] is not None:
        outs["dgate"] = (db * u * sig * (1 + z * (1 - sig))).to(t)
    du = db * act
    dyh = du * w1 if w1 is not None else du
    outs["dy"] = (_normed_back(dyh, yh, yr, s["post"]) if yr is not None else dyh).to(t)
    for name, grad in (("post_w", lambda: du * yh), ("post_b", lambda: du), ("pre_w", lambda: dn * hh),
                       ("pre_b", lambda: dn)):
        if s[name] is not None:
            outs["d" + name] = grad().sum((0, 1), dtype=torch.float64).float()
    return outs


# ---- the definition in 64 bits -----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("block_norm"):
        return _block_norm_exact(s, case["op"] == "block_norm_train")
    return _gated_exact(s)


def _gated_exact(s):
    """The recurrence row by row; the gradients with the state's gradient D run from the last row:
    dq = scale S do, dk = D v, dv = D^T k, dg = <D, a S_{t-1}>."""
    step, train = s["op"] == "gated_step", s["op"] == "gated_train"
    q, k, v = (s[n].double().unsqueeze(2) if step else s[n].double() for n in "qkv")
    B, H, L, dk = q.shape
    Hk, dv = k.shape[1], v.shape[-1]
    if train and B * H * L * dk * dv * 8 > 40e9:
        return None
    head = s["g"].dim() == 1
    g = s["g"].double()
    a = torch.exp(g[None, :, None].expand(B, H, L) if head else (g[..., None] if step else g))
    share = torch.arange(H, device=q.device) // (H // Hk)
    slots = None if s["slots"] is None else s["slots"].long()
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=q.device)
    if s["state0"] is not None:
        S = (s["state0"] if slots is None else s["state0"][slots]).double()
    n = torch.full((B,), L, device=q.device) if s["lengths"] is None else s["lengths"]
    live = (torch.arange(L, device=q.device) < n[:, None])[:, :, None, None, None]
    out = torch.zeros(B, H, L, dv, dtype=torch.float64, device=q.device)
    states = torch.empty(L + 1, B, H, dk, dv, dtype=torch.float64, device=q.device) if train else None
    full = bool((n == L).all())
    for i in range(L):
        if train:
            states[i] = S
        new = a[:, :, i, None, None] * S + k[:, share, i, :, None] * v[:, share, i, None, :]
        S = new if full else torch.where(live[:, i], new, S)
        o = s["scale"] * (q[:, :, i, None, :] @ S)[:, :, 0]
        out[:, :, i] = o if full else torch.where(live[:, i, :, 0], o, 0.0)
    if step:
        pool = s["state0"].double()
        if slots is None:
            pool = S
        else:
            pool[slots] = S
        return {"out": out[:, :, 0], "state": pool}
    last = S
    if slots is not None:
        last = s["state0"].double()
        last[slots] = S
    outs = {"out": out, "state": last}
    if not train:
        return outs
    states[L] = S
    do, D = s["scale"] * s["dout"].double(), s["dstate"].double()
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = torch.zeros(B, H, L, dtype=torch.float64, device=q.device)
    for i in reversed(range(L)):
        on = live[:, i]
        now = D + q[:, :, i, :, None] * do[:, :, i, None, :]
        now = now if full else torch.where(on, now, 0.0)
        dq[:, :, i] = torch.where(on[..., 0], (states[i + 1] @ do[:, :, i, :, None])[..., 0], 0.0)
        dkk[:, :, i].index_add_(1, share, (now @ v[:, share, i, :, None])[..., 0])
        dvv[:, :, i].index_add_(1, share, (k[:, share, i, None, :] @ now)[:, :, 0])
        back = a[:, :, i, None, None] * now
        dg[:, :, i] = (back * states[i]).sum((-1, -2))
        D = back if full else torch.where(on, back, D)
    outs |= {"dq": dq, "dk": dkk, "dv": dvv, "dg": dg.sum((0, 2)) if head else dg}
    return outs | ({"dstate0": D} if s["state0"] is not None else {})


def _block_norm_exact(s, train):
    """Forward from the definition, gradients by differentiating it."""
    leaves = {"d" + n: s[n].double().requires_grad_(train)
              for n in ("y", "r", "gate", "post_w", "post_b", "pre_w", "pre_b") if s[n] is not None}

    def norm(x, kind, w, b):
        if kind == "layer":
            x = x - x.sum(-1, keepdim=True) / x.shape[-1]
        if kind != "none":
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
        x = x * w if w is not None else x
        return x + b if b is not None else x

    u = norm(leaves["dy"], s["post"], leaves.get("dpost_w"), leaves.get("dpost_b"))
    if s["gate"] is not None:
        u = u * leaves["dgate"] / (1 + torch.exp(-leaves["dgate"]))
    h = s["residual_scale"] * leaves["dr"] + s["branch_scale"] * u
    n = norm(h, s["pre"], leaves.get("dpre_w"), leaves.get("dpre_b"))
    outs = {"h": h.detach(), "n": n.detach()}
    if train:
        grads = torch.autograd.grad((h, n), list(leaves.values()), (s["dh"].double(), s["dn"].double()))
        outs |= dict(zip(leaves, grads))
    return outs


# ---- what a pass cannot do without --------------------------------------------------------
def work(case):
    """Each input read once, each output written once; the operations of the formulas that no order of
    them saves: the state's update and its products with the rows."""
    op, z, B = case["op"], BYTES[case["dtype"]], case["B"]
    if op.startswith("block_norm"):
        E, zr = B * case["L"] * case["d"], BYTES[case["residual"]]
        vectors = sum(((case["post"] == "layer") + 1, (case["pre"] == "layer") + 1)) if case["affine"] else 0
        n = E * ((3 if case["gated"] else 2) * z + 2 * zr) + 4 * vectors * case["d"]
        if op == "block_norm":
            return {"bytes": n, "flops": 20 * E}
        return {"bytes": n + E * ((3 if case["gated"] else 2) * z + 2 * zr) + 4 * vectors * case["d"],
                "flops": 70 * E}
    H, Hk, dk, dv, L = case["H"], case["Hk"], case["dk"], case["dv"], case.get("L", 1)
    qo, kv, state = B * H * L * (dk + dv) * z, B * Hk * L * (dk + dv) * z, 4 * B * H * dk * dv
    gates = 4 * H * (B * L if case["gates"] == "token" else 1)
    one = 2 * B * H * L * dk * dv
    first = op == "gated_step" or case["initial"] or case.get("slots")
    n = qo + kv + gates + state * (2 if first else 1)
    if op != "gated_train":
        return {"bytes": n, "flops": 2 * one}
    return {"bytes": n + qo + kv + gates + state * (2 if first else 1), "flops": 7 * one}
