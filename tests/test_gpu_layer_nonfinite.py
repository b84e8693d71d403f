"""Infinities and NaN in the gated recurrence: a gate of 0 forgets them, and nothing else does.

Which entries are NaN, +inf and -inf is compared with the recurrence run row by row in 64 bits;
the finite rows before the first bad one are within the usual bounds."""
import numpy as np
import pytest

import layer_reference as ref
from test_gpu_layer import check, dev, host

pytestmark = pytest.mark.gpu


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


def forget(a, h):
    with np.errstate(invalid="ignore"):
        return np.where(a == 0, 0.0, a * h)


def forward(x, g, kind, complement, h0):
    """(out, state before each row, last), a gate of 0 forgetting everything."""
    a, w, _ = ref.gates(kind, g, complement)
    h = np.zeros(x[:, :, 0].shape) if h0 is None else h0
    out, before = np.empty_like(x), np.empty_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(x.shape[2]):
            before[:, :, t] = h
            h = forget(a[:, :, t], h) + w[:, :, t] * x[:, :, t]
            out[:, :, t] = h
    return out, before, h


def backward(x, g, dout, before, kind, complement):
    """(dx, dg, dh0); where da/dg is 0 so is dg."""
    a, w, slope = ref.gates(kind, g, complement)
    carry, e = np.zeros(x[:, :, 0].shape), np.empty_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in reversed(range(x.shape[2])):
            e[:, :, t] = dout[:, :, t] + carry
            carry = forget(a[:, :, t], e[:, :, t])
        dg = e * slope * (before - x if complement else before)
        return e * w, dg if kind == "value" else np.where(slope == 0, 0.0, dg), carry


KINDS = {"NaN": np.isnan, "+inf": np.isposinf, "-inf": np.isneginf}


def same_kind(name, got, want, kinds=None):
    """NaN, +inf, -inf and so finite values in the same places."""
    got = host(got).reshape(want.shape)
    for what, where in (kinds or KINDS).items():
        wrong = np.argwhere(where(got) != where(want))
        assert not len(wrong), f"{name}: {what} in other places, first {wrong[0]}, {len(wrong)} in all"


# the sign of an infinite gradient of the gate is that of h - x, which may be a rounding apart from 0
UNSIGNED = {"NaN": np.isnan, "infinity": np.isinf}
# an infinite gate makes infinities of either sign, whose sums NaN depend on how rows are grouped
FINITE = {"finite": np.isfinite}


def steady(kind, a):
    """The gate input of a gate a."""
    return {"value": a, "log": np.log(a), "sigmoid": np.log(a / (1 - a))}[kind]


# A run of rows is combined through the product of its gates, which is 0 in fp32 although no gate is:
# (shape, gate): 2048 rows in a cluster, tiles of 128 or 256 rows; enough heads for no cluster, 16 rows
# at a time, with fp32 and bf16 activations
UNDERFLOWING = [((1, 2, 2048, 64), 0.44), ((2, 80, 300, 64), 0.001), ((2, 80, 131, 34), 1e-20)]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("shape,gate", UNDERFLOWING, ids=str)
@pytest.mark.parametrize("kind", ["value", "log", "sigmoid"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
def test_small_gates_do_not_forget(la, shape, gate, kind, complement, dtype, gate_dtype):
    rng = np.random.default_rng(20)
    B, H, L, d = shape
    x, g = rng.normal(size=shape), np.full(shape, steady(kind, gate))
    row = min(100, L // 3)
    x[0, 0, row], x[-1, -1, row] = np.nan, -np.inf
    tx, tg = dev(x, dtype), dev(g, gate_dtype)
    hx, hg = host(tx), host(tg)
    want, before, last = forward(hx, hg, kind, complement, None)
    assert np.isnan(last[0, 0]).all() and np.isneginf(last[-1, -1]).all()
    kw = dict(gate_kind=kind, complement=complement)
    out, got_last, chunks = la.recurrence_fwd(tx, tg, save_chunks=True, **kw)
    same_kind("out", out, want)
    same_kind("last", got_last, last)
    same_kind("chunks", chunks, before[:, :, ::la.LA_RECURRENCE_CHUNK])
    bound = ref.recurrence_bounds(hx[:, :, :row], hg[:, :, :row], kind, complement)
    check("rows before", out[:, :, :row], want[:, :, :row], bound, dtype)
    # from the state before row 0
    h0 = rng.normal(size=(B, H, d))
    h0[0, 0], h0[-1, -1] = np.inf, np.nan
    clean = rng.normal(size=shape)
    tx = dev(clean, dtype)
    want, _, last = forward(host(tx), hg, kind, complement, host(dev(h0)))
    out, got_last = la.recurrence_fwd(tx, tg, h0=dev(h0), **kw)
    same_kind("out from h0", out, want)
    same_kind("last from h0", got_last, last)
    # backwards
    dout = rng.normal(size=shape)
    dout[0, 0, L - 1 - row], dout[-1, -1, L - 1 - row] = np.nan, np.inf
    td = dev(dout, dtype)
    _, before, _ = forward(host(tx), hg, kind, complement, None)
    wx, wg, w0 = backward(host(tx), hg, host(td), before, kind, complement)
    chunks = la.recurrence_fwd(tx, tg, save_chunks=True, **kw)[2]
    dx, dg, dh0 = la.recurrence_bwd(tx, tg, chunks, td, **kw)
    same_kind("dx", dx, wx)
    same_kind("dg", dg, wg, UNSIGNED)
    same_kind("dh0", dh0, w0)


@pytest.mark.parametrize("kind", ["log", "sigmoid"])
@pytest.mark.parametrize("g", [-88.0, -100.0, -300.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_below_the_normal_range_do_not_forget(la, kind, g, dtype):
    """exp(-100) is not 0, though fp32 has no normal number for it."""
    rng = np.random.default_rng(21)
    for shape in ((1, 2, 700, 64), (2, 80, 40, 64)):
        L = shape[2]
        x, gate = rng.normal(size=shape), np.full(shape, 2.0 if kind == "sigmoid" else -0.1)
        gate[:, :, L // 2] = g
        x[0, 0, 3], x[-1, -1, 3] = np.inf, np.nan
        tx, tg = dev(x, dtype), dev(gate, dtype)
        want, _, last = forward(host(tx), host(tg), kind, False, None)
        out, got_last = la.recurrence_fwd(tx, tg, gate_kind=kind)
        same_kind("out", out, want)
        same_kind("last", got_last, last)
        state = dev(want[:, :, L // 2 - 1])
        step = la.recurrence_step(tx[:, :, L // 2].contiguous(), tg[:, :, L // 2].contiguous(), state, gate_kind=kind)
        same_kind("step", step, want[:, :, L // 2])
        same_kind("state", state, want[:, :, L // 2])


def test_complement_below_the_normal_range(la):
    """1 - a of a logit of 100 is not 0 either: an infinite input comes through, and its gradient."""
    rng = np.random.default_rng(23)
    for shape in ((1, 2, 700, 64), (2, 80, 40, 64)):
        x, g, dout = rng.normal(size=shape), np.full(shape, 2.0), rng.normal(size=shape)
        row = shape[2] // 2
        g[:, :, row] = 100.0
        x[0, 0, row], dout[-1, -1, row] = np.inf, -np.inf
        x, dout = host(dev(x)), host(dev(dout))
        want, before, _ = forward(x, g, "sigmoid", True, None)
        out, _, chunks = la.recurrence_fwd(dev(x), dev(g), complement=True, save_chunks=True)
        same_kind("out", out, want)
        wx, wg, w0 = backward(x, g, dout, before, "sigmoid", True)
        dx, dg, dh0 = la.recurrence_bwd(dev(x), dev(g), chunks, dev(dout), complement=True)
        same_kind("dx", dx, wx)
        same_kind("dg", dg, wg, UNSIGNED)
        same_kind("dh0", dh0, w0)
        step = la.recurrence_step(dev(x[:, :, row]), dev(g[:, :, row]), dev(before[:, :, row]), complement=True)
        same_kind("step", step, want[:, :, row])


@pytest.mark.parametrize("row", [0, 2, 16, 130])
@pytest.mark.parametrize("apart", [1, 11, 200])
@pytest.mark.parametrize("kind,bad", [("value", np.nan), ("value", np.inf), ("log", np.nan), ("log", np.inf),
                                      ("sigmoid", np.nan)])
def test_gate_zero_forgets_a_bad_gate(la, row, apart, kind, bad):
    """A NaN or infinite gate reaches no row from the next gate of 0 on; backwards no row before it."""
    rng = np.random.default_rng(22)
    kinds = KINDS if np.isnan(bad) else FINITE
    for shape, dtype in (((1, 2, 600, 64), "f32"), ((2, 80, 350, 34), "f32"), ((2, 80, 350, 34), "bf16")):
        L, zero = shape[2], row + apart
        x, g = rng.normal(size=shape), np.full(shape, steady(kind, 0.9))
        g[:, :, row], g[:, :, zero] = bad, 0.0 if kind == "value" else -np.inf
        tx, tg = dev(x, dtype), dev(g, dtype)
        hx, hg = host(tx), host(tg)
        want, before, last = forward(hx, hg, kind, False, None)
        out, got_last, chunks = la.recurrence_fwd(tx, tg, gate_kind=kind, save_chunks=True)
        same_kind("out", out, want, kinds)
        same_kind("last", got_last, last, kinds)
        same_kind("chunks", chunks, before[:, :, ::la.LA_RECURRENCE_CHUNK], kinds)
        tail = ref.recurrence_bounds(hx[:, :, zero:], hg[:, :, zero:], kind, False)
        check("rows behind", out[:, :, zero:], want[:, :, zero:], tail, dtype)
        # backwards: the bad gate behind the zero one
        g[:, :, row], g[:, :, zero] = g[:, :, zero].copy(), bad
        tg = dev(g, dtype)
        do = dev(rng.normal(size=shape), dtype)
        want, before, _ = forward(hx, host(tg), kind, False, None)
        wx, wg, w0 = backward(hx, host(tg), host(do), before, kind, False)
        chunks = la.recurrence_fwd(tx, tg, gate_kind=kind, save_chunks=True)[2]
        dx, dg, dh0 = la.recurrence_bwd(tx, tg, chunks, do, gate_kind=kind)
        same_kind("dx", dx, wx, kinds)
        same_kind("dg", dg, wg, kinds)
        same_kind("dh0", dh0, w0, kinds)
