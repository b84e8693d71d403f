"""Plain 64-bit forms of the operators around the attention (recurrence, rotary positions,
group norm), written from their formulas, with bounds on what an fp32 evaluation that rounds
its result once may be off.  numpy only; shapes [B, H, L, d].

u = 2^-24 is the unit roundoff of fp32; half_step(dtype) that of the stored type.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 2.0 ** -126  # smallest normal number of both types: what rounds below it is off by less


def gates(kind, g, complement):
    """(a, w, da/dg) in 64 bits."""
    g = g.astype(np.float64)
    with np.errstate(over="ignore"):
        if kind == "value":
            a, c, slope = g, 1.0 - g, np.ones_like(g)
        elif kind == "log":
            a, c = np.exp(g), -np.expm1(g)
            slope = a
        else:
            a, c = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
            slope = a * c
    return a, (c if complement else np.ones_like(a)), slope


def recurrence(x, g, kind, complement, h0=None, lengths=None):
    """(out, last, states before each row) row by row."""
    a, w, _ = gates(kind, g, complement)
    B, H, L, d = x.shape
    h = np.zeros((B, H, d)) if h0 is None else h0.astype(np.float64).copy()
    out, before = np.zeros((B, H, L, d)), np.zeros((B, H, L, d))
    for t in range(L):
        before[:, :, t] = h
        for b in range(B):
            if lengths is None or t < lengths[b]:
                h[b] = a[b, :, t] * h[b] + w[b, :, t] * x[b, :, t]
                out[b, :, t] = h[b]
    return out, h, before


def recurrence_grads(x, g, dout, dlast, kind, complement, h0=None, lengths=None):
    """(dx, dg, dh0, e): e_t = dout_t + a_{t+1} e_{t+1}."""
    a, w, slope = gates(kind, g, complement)
    _, _, before = recurrence(x, g, kind, complement, h0, lengths)
    B, H, L, d = x.shape
    carry = np.zeros((B, H, d)) if dlast is None else dlast.astype(np.float64).copy()
    e = np.zeros((B, H, L, d))
    for t in reversed(range(L)):
        for b in range(B):
            if lengths is None or t < lengths[b]:
                e[b, :, t] = dout[b, :, t] + carry[b]
                carry[b] = a[b, :, t] * e[b, :, t]
    dg = e * slope * (before - x if complement else before)
    return e * w, dg, carry, e


# ---- bounds of the recurrence ----------------------------------------------------------
# A gate a, and 1 - a, evaluated in fp32 is off by at most K = (9 + 1.3 |g|) u relatively: the
# argument g log2(e) of a power of two is rounded twice (1.3 |g| u), the power is good to 4 u, a
# sum 1 u, a reciprocal 2 u, a product or difference 2 u (value gates: 1 u).  A row multiplies by
# its gate and adds, 2 u more, and where rows are combined in groups a product of gates has as
# many factors and a combination one product and one sum: every row that a term passes
# multiplies it by (1 + K + 2 u) at most.  A term enters with w x: K + 2 u, and the groups'
# combinations add 4 u.  So the error of h_t is at most  sum_s (sum_{s<r<=t} (K_r + 2 u) +
# K_s + 6 u) |w_s x_s| prod a  =  N_t,  with
#     N_t = a (N_{t-1} + (K_t + 2 u) M_{t-1}) + (K_t + 6 u) |w x|,   M_t = a M_{t-1} + |w x|.
# Products of gates below the normal range are flushed or rounded absolutely: TINY a row.
def gate_error(kind, g):
    if kind == "value":
        return np.full(g.shape, U)
    return U * (9 + 1.3 * np.minimum(np.abs(g.astype(np.float64)), 200.0))


def recurrence_bounds(x, g, kind, complement, h0=None, lengths=None):
    """Error bound of h after each row, in fp32 (no rounding to the stored type)."""
    a, w, _ = gates(kind, g, complement)
    K, terms = gate_error(kind, g), np.abs(w * x)
    a = np.abs(a)
    B, H, L, d = x.shape
    M = np.zeros((B, H, d)) if h0 is None else np.abs(h0.astype(np.float64))
    N, out = np.zeros((B, H, d)), np.zeros_like(terms)
    for t in range(L):
        for b in range(B):
            if lengths is None or t < lengths[b]:
                N[b] = a[b, :, t] * (N[b] + (K[b, :, t] + 2 * U) * M[b]) + (K[b, :, t] + 6 * U) * terms[b, :, t]
                M[b] = a[b, :, t] * M[b] + terms[b, :, t]
        out[:, :, t] = N
    return out + TINY * np.arange(1, L + 1)[:, None]


def recurrence_grad_bounds(x, g, dout, dlast, kind, complement, h0=None, lengths=None):
    """(bound of dx, of dg, of dh0) in fp32.  e runs the same recurrence backwards, so it has the
    same bound; dx = w e adds K + 1 u; dg = e slope (before - x) adds the bounds of its factors,
    2 K + 1 u of the slope and 3 u of the operations."""
    a, w, slope = gates(kind, g, complement)
    K, a = gate_error(kind, g), np.abs(a)
    B, H, L, d = x.shape
    _, _, before = recurrence(x, g, kind, complement, h0, lengths)
    hb = np.zeros_like(before)
    full = recurrence_bounds(x, g, kind, complement, h0, lengths)
    hb[:, :, 1:] = full[:, :, :-1]
    _, _, dh0, e = recurrence_grads(x, g, dout, dlast, kind, complement, h0, lengths)
    eb, terms = np.zeros_like(before), np.abs(dout)
    M = np.zeros((B, H, d)) if dlast is None else np.abs(dlast.astype(np.float64))
    N = np.zeros((B, H, d))
    for t in reversed(range(L)):
        for b in range(B):
            if lengths is None or t < lengths[b]:
                M[b] = M[b] + terms[b, :, t]
                N[b] = N[b] + 6 * U * terms[b, :, t]
                eb[b, :, t] = N[b]
                N[b] = a[b, :, t] * (N[b] + (K[b, :, t] + 2 * U) * M[b])
                M[b] = a[b, :, t] * M[b]
    eb += TINY * L
    factor = before - x if complement else before
    dxb = np.abs(w) * eb + (K + 2 * U) * np.abs(e * w)
    dgb = np.abs(slope) * (eb * np.abs(factor) + (np.abs(e) + eb) * (hb + U * np.abs(factor)))
    dgb += (2 * K + 4 * U) * np.abs(e * slope * factor)
    return dxb, dgb, N + 2 * U * np.abs(dh0) + TINY * L


def stored(bound, ref, dtype):
    """The bound with the rounding to the stored type."""
    return bound * (1 + HALF_STEP[dtype]) + HALF_STEP[dtype] * np.abs(ref) + TINY


# ---- rotary positions --------------------------------------------------------------------
def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, fast=32.0, slow=1.0):
    out = []
    for j in range(rot // 2):
        theta = base ** (-2.0 * j / rot)
        if scaling == "linear":
            theta /= factor
        elif scaling == "parts":
            keep = min(1.0, max(0.0, (original * theta / (2 * np.pi) - slow) / (fast - slow)))
            theta = theta * keep + theta / factor * (1.0 - keep)
        out.append(theta)
    return np.array(out)


def rotary(x, positions, theta, layout, inverse=False, amplitude=1.0):
    """x [B,H,L,d], positions [B,L] -> (rotated, bound in fp32).

    A sine or cosine is off by at most 4 u (angle below an eighth of a turn off by a rounding:
    0.8 u; the function 2 u; the table 2^-33 of a turn, below 0.02 u), the amplitude's product
    by 1 u more, the two products and their sum by 2 u: 8 u (|u| + |v|) amplitude in all.  The
    64-bit angle itself is off by 2^-52 of its size."""
    rot = 2 * len(theta)
    y, bound = x.astype(np.float64).copy(), np.zeros(x.shape)
    angle = positions.astype(np.float64)[:, None, :, None] * theta
    c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
    if layout == "half":
        i, j = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    u, v = x[..., i].astype(np.float64), x[..., j].astype(np.float64)
    y[..., i], y[..., j] = amplitude * (u * c - v * s), amplitude * (u * s + v * c)
    b = abs(amplitude) * (np.abs(u) + np.abs(v)) * (8 * U + np.abs(angle) * 2.0 ** -51)
    bound[..., i], bound[..., j] = b, b
    return y, bound


# ---- group norm --------------------------------------------------------------------------
def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def group_norm(x, w, b, gate, eps, act, center, dout=None):
    """x [B,H,L,d]; w, b [H,d] or None; gate, dout [B,L,H,d] or None.  A dict of the outputs in
    64 bits ([B,L,H,d]; dw, db [H,d]) and of their bounds in fp32.

    With c = (d + 8) u the relative bound of a sum of d values: the mean is off by c mean|x|,
    a centred value by that and 1 u, which rstd scales: dxh = rstd (c mean|x| + 2 u |xc|); rstd
    by half the variance's relative error, mean(dxc |xc|) / var + c + 8 u.  With k = (8 + 2.5 |z|)
    u the sigmoid s is off by at most k s (its argument is scaled and rounded, 2.4 |z| u, the
    power 4 u, the sum 1 u, the quotient 2 u), so z s by k |z s| + 1 u and the slope s + z s (1 - s)
    by k (s + 2 |z s|) + 4 u (s + |z s|); the error of z comes in by slopes of at most 1.1 and
    0.5."""
    x = np.swapaxes(x.astype(np.float64), 1, 2)
    d = x.shape[-1]
    c = (d + 8) * U
    w = np.ones(x.shape[2:]) if w is None else w.astype(np.float64)
    b = np.zeros(x.shape[2:]) if b is None else b.astype(np.float64)
    mean = x.mean(-1, keepdims=True) if center else np.zeros(x.shape[:-1] + (1,))
    xc = x - mean
    rstd = 1.0 / np.sqrt((xc * xc).mean(-1, keepdims=True) + eps)
    xh = xc * rstd
    dxc = (c * np.abs(x).mean(-1, keepdims=True) if center else 0.0) + U * np.abs(xc)
    rel = (dxc * np.abs(xc)).mean(-1, keepdims=True) * rstd ** 2 + c + 8 * U
    xh_b = rstd * dxc + np.abs(xh) * (rel + 2 * U)
    y = xh * w + b
    y_b = np.abs(w) * xh_b + 2 * U * (np.abs(xh * w) + np.abs(b))
    z = y if gate is None else gate.astype(np.float64)
    z_b = y_b if gate is None else np.zeros_like(z)
    if act == "silu":
        sg = _sigmoid(z)
        f, slope = z * sg, sg * (1 + z * (1 - sg))
        k = U * (8 + 2.5 * np.minimum(np.abs(z), 200.0))
        f_b = 1.1 * z_b + (k + U) * np.abs(f)
        slope_b = 0.5 * z_b + k * (sg + 2 * np.abs(f)) + 4 * U * (sg + np.abs(f))
    else:
        f, slope, f_b, slope_b = z, np.ones_like(z), z_b, np.zeros_like(z)
    out = f if gate is None else y * f
    out_b = f_b if gate is None else y_b * np.abs(f) + np.abs(y) * f_b + y_b * f_b + 2 * U * np.abs(out)
    res = {"out": (out, out_b)}
    if dout is None:
        return res
    do = dout.astype(np.float64)
    if gate is None:
        dy, dy_b = do * slope, np.abs(do) * slope_b
    else:
        dy, dy_b = do * f, np.abs(do) * f_b
        dgate = do * y * slope
        res["dgate"] = (dgate, np.abs(do) * (y_b * np.abs(slope) + np.abs(y) * slope_b + y_b * slope_b)
                        + 3 * U * np.abs(dgate))
    dy_b = dy_b + 2 * U * np.abs(dy)
    n = do.shape[0] * do.shape[1]
    # summed in groups whose partial sums are summed: at most n roundings for a term
    res["dw"] = ((dy * xh).sum((0, 1)), (np.abs(dy) * xh_b + dy_b * np.abs(xh) + dy_b * xh_b).sum((0, 1))
                 + (n + 2) * U * np.abs(dy * xh).sum((0, 1)))
    res["db"] = (dy.sum((0, 1)), dy_b.sum((0, 1)) + n * U * np.abs(dy).sum((0, 1)))
    e, e_b = dy * w, dy_b * np.abs(w) + U * np.abs(dy * w)

    def mean_with_bound(v, v_b):
        return v.mean(-1, keepdims=True), v_b.mean(-1, keepdims=True) + c * np.abs(v).mean(-1, keepdims=True)

    m1, m1_b = mean_with_bound(e, e_b) if center else (0.0, 0.0)
    m2, m2_b = mean_with_bound(e * xh, np.abs(e) * xh_b + e_b * np.abs(xh) + e_b * xh_b)
    inner = e - m1 - xh * m2
    inner_b = e_b + m1_b + xh_b * np.abs(m2) + np.abs(xh) * m2_b + xh_b * m2_b
    inner_b = inner_b + 3 * U * (np.abs(e) + np.abs(m1) + np.abs(xh * m2))
    res["dx"] = (inner * rstd, rstd * (inner_b * (1 + rel + 2 * U) + np.abs(inner) * (rel + 2 * U)))
    return res
