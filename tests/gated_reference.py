"""The gated attention and the norms around a block in 64 bits, row by row, on the CPU, and what their
tests draw and allow."""
import torch

U = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def shared(x, H):
    """[B, Hk, ...] repeated for the H / Hk heads of each key head."""
    return x.repeat_interleave(H // x.shape[1], 1)


def gates(g, B, H, L):
    """log decays [H] or [B, H, L] as [B, H, L]."""
    g = g.double()
    return g[None, :, None].expand(B, H, L) if g.dim() == 1 else g


def forward(q, k, v, g, scale, state0=None, lengths=None, keep=False):
    """(out, state[, states before every row and behind the last]) of the recurrence."""
    B, H, L, d = q.shape
    q, k, v = q.double(), shared(k.double(), H), shared(v.double(), H)
    a = torch.exp(gates(g, B, H, L))
    n = [L] * B if lengths is None else [max(0, min(L, int(x))) for x in lengths]
    S = torch.zeros(B, H, d, v.shape[-1], dtype=torch.float64) if state0 is None else state0.double().clone()
    out = torch.zeros(B, H, L, v.shape[-1], dtype=torch.float64)
    states = [S.clone()]
    for t in range(L):
        on = torch.tensor([t < x for x in n])[:, None, None]
        old = torch.where(a[:, :, t, None, None] == 0, 0.0, a[:, :, t, None, None] * S)
        new = old + k[:, :, t, :, None] * v[:, :, t, None, :]
        S = torch.where(on[..., None], new, S)
        out[:, :, t] = torch.where(on, scale * (q[:, :, t, None, :] @ S)[:, :, 0], 0.0)
        if keep:
            states.append(S.clone())
    return (out, S, states) if keep else (out, S)


def backward(q, k, v, g, dout, scale, state0=None, lengths=None, dstate=None):
    """dict of the gradients, with the state's gradient D run from the last row."""
    B, H, L, d = q.shape
    Hk, e = k.shape[1], v.shape[-1]
    states = forward(q, k, v, g, scale, state0, lengths, keep=True)[2]
    q, k, v, do = q.double(), shared(k.double(), H), shared(v.double(), H), dout.double()
    a = torch.exp(gates(g, B, H, L))
    n = [L] * B if lengths is None else [max(0, min(L, int(x))) for x in lengths]
    D = torch.zeros(B, H, d, e, dtype=torch.float64) if dstate is None else dstate.double().clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = torch.zeros(B, H, L, dtype=torch.float64)
    for t in reversed(range(L)):
        on = torch.tensor([t < x for x in n])[:, None, None]
        now = D + scale * q[:, :, t, :, None] * do[:, :, t, None, :]
        dq[:, :, t] = torch.where(on, scale * (states[t + 1] @ do[:, :, t, :, None])[..., 0], 0.0)
        dk[:, :, t] = torch.where(on, (now @ v[:, :, t, :, None])[..., 0], 0.0)
        dv[:, :, t] = torch.where(on, (k[:, :, t, None, :] @ now)[:, :, 0], 0.0)
        back = torch.where(a[:, :, t, None, None] == 0, 0.0, a[:, :, t, None, None] * now)
        dg[:, :, t] = torch.where(on[..., 0], (back * states[t]).sum((-1, -2)), 0.0)
        D = torch.where(on[..., None], back, D)
    join = lambda x: x.unflatten(1, (Hk, H // Hk)).sum(2)  # noqa: E731
    return dict(dq=dq, dk=join(dk), dv=join(dv), dg=dg if g.dim() == 3 else dg.sum((0, 2)), dstate0=D)


def magnitudes(q, k, v, g, scale, state0, lengths, dout=None, dstate=None):
    """The same sums with every term's absolute value: what roundings are relative to."""
    args = (q.abs(), k.abs(), v.abs(), g)
    s0 = None if state0 is None else state0.abs()
    out, state = forward(*args, abs(scale), s0, lengths)
    m = dict(out=out, state=state)
    if dout is not None:
        m |= backward(*args, dout.abs(), abs(scale), s0, lengths, None if dstate is None else dstate.abs())
        m["end"] = torch.zeros(state.shape[:2], dtype=torch.float64) if dstate is None else (state * dstate.abs()).sum((-1, -2))
    return m


def close(name, got, want, size, dtype, steps, rows=None):
    """got against the 64-bit value.  In fp32 every term meets at most `steps` roundings of U on its way
    (decays, products, sums), so no value is off by more than steps U of its terms' magnitude `size`, and
    with independent roundings the root mean square by sqrt(steps) U of theirs.  Where operands of the
    matrix instructions are rounded to bf16 (dtype bf16) each product is off by another half step: at most
    2^-8 of the magnitude for the row's pairs and 2^-8 for the state they are added to; three independent
    roundings of half a step, uniform, are 2^-8 of the result in the root mean square."""
    got, want, size = got.double().cpu(), want.double(), size.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), name
    err = (got - want).abs()
    half = HALF[dtype]
    most = steps * U * size + half * want.abs()
    if dtype == torch.bfloat16:
        most = most + 2 * half * size
    bad = err > most + 1e-37
    assert not bad.any(), (name, int(bad.sum()), float((err - most).max()), float(err.max()))
    rms = lambda x: float(x.square().mean().sqrt())  # noqa: E731
    allowed = (steps ** 0.5) * U * rms(size) + (half * rms(want) if dtype == torch.bfloat16 else U * rms(want))
    assert rms(err) <= allowed + 1e-37, (name, rms(err), allowed, rms(want))


def draw(B, H, Hk, L, d, e, dtype, kind="token", initial=False, padded=False, seed=0, resets=0.02):
    """Inputs on the CPU: q, k, v, g, state0, lengths, dout, dstate."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, v = n(B, H, L, d).to(dtype), n(B, Hk, L, d).to(dtype), n(B, Hk, L, e).to(dtype)
    if kind == "head":
        g = torch.log1p(-torch.exp2(-2.0 - 8.0 * torch.rand(H, generator=gen)))
    else:
        g = -torch.nn.functional.softplus(1.5 * n(B, H, L) - 2.0)
        g = g.masked_fill(torch.rand(B, 1, L, generator=gen) < resets, float("-inf"))
    state0 = n(B, H, d, e) if initial else None
    lengths = None
    if padded:
        lengths = torch.randint(0, L + 1, (B,), generator=gen, dtype=torch.int32)
        lengths[0] = L
        if B > 1:
            lengths[1] = 0
        if B > 2:
            lengths[2] = max(1, L - 3)
    return q, k, v, g, state0, lengths, n(B, H, L, e).to(dtype), n(B, H, d, e)
