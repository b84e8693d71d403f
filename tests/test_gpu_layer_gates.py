"""How exact the recurrence's gates are: a and 1 - a read off single rows, over the whole range of the
gate input, and a long memory with a steady gate.

u = 2^-24.  For fp32 activations (FINE in the kernel):
  sigmoid  the smaller of a and 1 - a is e / (1 + e): the power 4 u, its argument's rest multiplied in
           1 u, the sum 1 u, the reciprocal 2 u, the product 1 u: 9 u relatively.  The larger is 1
           less that one: half a step below 1 (u / 2) and 9 u of the smaller.
  log      below log 2, with 1 - a asked for: the series' value 1 u, s and q and their product 3 u, what
           the series leaves out 0.4 u: 6 u of 1 - a, and a is 1 less it: u / 2 and 6 u of 1 - a.
           Without it, below 1/16: u / 2, the inner terms' 2 u |g|, the series' rest |g|^5 / 100.
           Elsewhere a is off by (4 + 1.3 |g|) u relatively: 2^x 4 u, its argument g log2(e) rounded
           twice (the constant and the product, 1.3 |g| u).
For bf16 activations every gate is off by (9 + 1.3 |g|) u at most, as the kernel says.  What is below
the normal range is flushed: TINY."""
import numpy as np
import pytest

import layer_reference as ref
from test_gpu_layer import check, dev, host

pytestmark = pytest.mark.gpu

U, TINY = ref.U, ref.TINY


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunkwise_causal_linear_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def la():
    import chunkwise_causal_linear_gb300 as la
    return la


def inputs(kind, rng, n):
    """n gate inputs, even over the logarithm of their size from 1e-7 to 80, of either sign for logits."""
    m = np.exp(rng.uniform(np.log(1e-7), np.log(80.0), n))
    return -m if kind == "log" else m * rng.choice([-1.0, 1.0], n)


def read_gates(la, kind, g, dtype, complement):
    """(a, 1 - a or None) of one row: from a state of 1 and no input, and from no state and an input of 1."""
    import torch
    shape = (1, g.numel() // 64, 1, 64)
    g = g.view(shape)
    zero = torch.zeros(shape, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    h0 = torch.ones(1, shape[1], 64, device="cuda")
    kw = dict(gate_kind=kind, complement=complement)
    a = la.recurrence_fwd(zero, g, h0=h0, **kw)[1]
    # the decoding step has the same gates
    la.recurrence_step(zero[:, :, 0], g[:, :, 0], h0, **kw)
    assert torch.equal(a, h0)
    if not complement:
        return host(a).ravel(), None
    return host(a).ravel(), host(la.recurrence_fwd(zero + 1, g, **kw)[1]).ravel()


def close(name, got, want, bound, g):
    off = np.abs(got - want) - bound
    i = np.argmax(off)
    assert off[i] <= 0, f"{name} at {g[i]!r}: off by {abs(got[i] - want[i]) / U:.2f} u, bound {bound[i] / U:.2f} u"


@pytest.mark.parametrize("gate_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("complement", [False, True])
def test_sigmoid_gates(la, gate_dtype, complement):
    t = dev(inputs("sigmoid", np.random.default_rng(40), 64 * 2048), gate_dtype)
    g = host(t)
    want_a, want_c = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    a, c = read_gates(la, "sigmoid", t, "f32", complement)
    less = np.minimum(want_a, want_c)
    for name, got, want in (("a", a, want_a), ("1 - a", c, want_c)):
        if got is not None:
            close(name, got, want, np.where(want < 0.5, 9 * U * less, U / 2 + 9 * U * less) + TINY, g)
    if complement:  # the two go together: 1 less the other, rounded
        assert np.abs(a + c - 1).max() <= U / 2


@pytest.mark.parametrize("gate_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("complement", [False, True])
def test_log_gates(la, gate_dtype, complement):
    t = dev(inputs("log", np.random.default_rng(41), 64 * 2048), gate_dtype)
    g = host(t)
    want_a, want_c, m = np.exp(g), -np.expm1(g), np.abs(g)
    a, c = read_gates(la, "log", t, "f32", complement)
    far = U * (4 + 1.3 * m) * want_a + TINY
    if complement:
        close("a", a, want_a, np.where(m < 0.693, U / 2 + 6 * U * want_c, far), g)
        close("1 - a", c, want_c, np.where(m < 0.693, 6 * U * want_c, far + U), g)
        assert np.abs(a + c - 1).max() <= 1.5 * U
    else:
        close("a", a, want_a, np.where(m < 0.0625, U / 2 + 2 * U * m + m ** 5 / 100, far), g)


@pytest.mark.parametrize("kind", ["log", "sigmoid"])
@pytest.mark.parametrize("gate_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("complement", [False, True])
def test_gates_of_bf16_activations(la, kind, gate_dtype, complement):
    t = dev(inputs(kind, np.random.default_rng(42), 64 * 2048), gate_dtype)
    g = host(t)
    want_a, want_c, _ = ref.gates(kind, g, True)
    a, c = read_gates(la, kind, t, "bf16", complement)
    for name, got, want in (("a", a, want_a), ("1 - a", c, want_c)):
        if got is not None:
            close(name, got, want, ref.gate_error("log", g) * want + TINY, g)


@pytest.mark.parametrize("kind,g", [("log", -1e-4), ("sigmoid", 9.2)])
@pytest.mark.parametrize("gate_dtype", ["f32", "bf16"])
def test_steady_long_memory(la, kind, g, gate_dtype):
    """65536 rows that remember 10^4 of them: constant and random inputs, averaged (complement).

    A row's step is off by the gate's rounding, U / 2 and 9 u of 1 - a, by the 2 u of its product and
    sum, and by 16 u of what it adds (layer_reference's recurrence with that gate)."""
    rng = np.random.default_rng(43)
    shape = (1, 2, 65536, 32)
    x = rng.normal(size=shape)
    x[:, 0] = 1.0
    tx, tg = dev(x), dev(np.full(shape, g), gate_dtype)
    out, last = la.recurrence_fwd(tx, tg, gate_kind=kind, complement=True)
    hx, hg = host(tx), host(tg)
    want, wlast, _ = ref.recurrence(hx, hg, kind, True)
    a, w, _ = (v[0, 0, 0, 0] for v in ref.gates(kind, hg[:, :, :1, :1], True))
    N, M, bound = np.zeros((1, 2, 32)), np.zeros((1, 2, 32)), np.empty(shape)
    for t in range(shape[2]):
        terms = np.abs(w * hx[:, :, t])
        N = a * N + (U / 2 + 9 * U * w + 2 * U) * M + 16 * U * terms
        M = a * M + terms
        bound[:, :, t] = N
    check("out", out, want, bound)
    check("last", last, wlast, N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
def test_silu_of_the_group_norm(la, dtype, gated):
    """SiLU and its slope over logits to 80: y is the bias where the weight is 0.

    fp32: the sigmoid s is off by 9 u relatively, f = z s by 10 u; the slope s + f (1 - s) by 9 u s, the
    error of 1 - s (9 u s and a rounding) times |f|, 10 u |f| (1 - s) and a rounding: 10 u (s + 2 |f|) in
    all.  bf16: (8 + 2.5 |z|) u in place of 9 u, and the rounding of the output.  A sigmoid below the
    normal range is 0."""
    import torch
    H, d, n = 64, 128, 64 * 128
    z = dev(inputs("sigmoid", np.random.default_rng(44), n), dtype)
    x = dev(np.random.default_rng(45).normal(size=(1, H, 1, d)), dtype)
    w, b = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda") if gated else z.float()
    gate = z.view(1, 1, n) if gated else None
    ones = torch.ones(1, 1, n, dtype=x.dtype, device="cuda")
    out = host(la.group_norm_fwd(x, w, b, gate=gate)).ravel()
    dx, dgate, dw, db = la.group_norm_bwd(x, ones, w, b, gate=gate)
    v = host(z)
    s, c = 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
    f, slope = v * s, s + v * s * c
    k = U * (9 if dtype == "f32" else 8 + 2.5 * np.abs(v))
    f_b = (k + U) * np.abs(f) + TINY * np.abs(v)
    slope_b = (k + U) * (s + 2 * np.abs(f)) + TINY * np.abs(v)
    close("out", out, f, ref.stored(f_b, f, dtype), v)
    # the gradient of the bias (y act(z) with a gate, act(y) without) is fp32 in either type
    close("dbias", host(db), f if gated else slope, f_b if gated else slope_b, v)
    if gated:  # dout y slope, y = 1
        close("dgate", host(dgate).ravel(), slope, ref.stored(slope_b + 3 * U * np.abs(slope), slope, dtype), v)
