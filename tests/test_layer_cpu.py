"""The operators around the attention, without a GPU: what their entry points refuse before
anything is launched, the rotary table, and the 64-bit forms that the GPU tests compare
against (gradients by central differences)."""
import ctypes

import numpy as np
import pytest

import chunkwise_causal_linear_gb300 as la
import layer_reference as ref
from chunkwise_causal_linear_gb300 import build as la_build

P = ctypes.c_void_p(1 << 20)  # never dereferenced: every call below fails on the host
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    la_build.build()
    return la.lib()


def st(b, h, l):
    return ctypes.byref(la.la_strides(b, h, l))


def rec_fwd(x=P, gate=P, h0=None, lengths=None, out=P, last=None, chunks=None, B=2, H=3, L=5, d=8, sx=None,
            sg=None, so=None, kind=0, comp=0, dtype=la.LA_F32, gdtype=la.LA_F32):
    return la.la_recurrence_fwd(x, gate, h0, lengths, out, last, chunks, B, H, L, d, sx, sg, so, kind, comp,
                                dtype, gdtype, None)


def rec_bwd(x=P, gate=P, chunks=P, lengths=None, dout=P, dlast=None, dx=P, dg=P, dh0=None, B=2, H=3, L=5, d=8,
            sx=None, sg=None, sdo=None, sdx=None, sdg=None, kind=0, comp=0, dtype=la.LA_F32, gdtype=la.LA_F32):
    return la.la_recurrence_bwd(x, gate, chunks, lengths, dout, dlast, dx, dg, dh0, B, H, L, d, sx, sg, sdo, sdx,
                                sdg, kind, comp, dtype, gdtype, None)


def rec_step(x=P, gate=P, state=P, out=P, B=2, H=3, d=8, kind=0, comp=0, dtype=la.LA_F32, gdtype=la.LA_F32):
    return la.la_recurrence_step(x, gate, state, out, B, H, d, kind, comp, dtype, gdtype, None)


def rotary(q=P, k=None, qo=P, ko=None, turns=P, pos=None, off=0, B=2, H=3, Hk=3, L=5, d=8, rot=8, sq=None,
           sk=None, sqo=None, sko=None, layout=0, inverse=0, amp=1.0, dtype=la.LA_F32):
    return la.la_rotary(q, k, qo, ko, turns, pos, off, B, H, Hk, L, d, rot, sq, sk, sqo, sko, layout, inverse,
                        amp, dtype, None)


def gn_fwd(x=P, w=None, b=None, gate=None, out=P, B=2, H=3, L=5, d=8, sx=None, sg=None, so=None, center=1,
           act=1, eps=1e-5, dtype=la.LA_F32):
    return la.la_group_norm_fwd(x, w, b, gate, out, B, H, L, d, sx, sg, so, center, act, eps, dtype, None)


def gn_bwd(x=P, w=None, b=None, gate=None, dout=P, dx=P, dgate=None, dw=None, db=None, B=2, H=3, L=5, d=8,
           sx=None, sg=None, sdo=None, sdx=None, sdg=None, center=1, act=1, eps=1e-5, dtype=la.LA_F32, ws=None,
           wsb=0):
    return la.la_group_norm_bwd(x, w, b, gate, dout, dx, dgate, dw, db, B, H, L, d, sx, sg, sdo, sdx, sdg, center,
                                act, eps, dtype, ws, wsb, None)


NULLS = [(rec_fwd, k) for k in ("x", "gate", "out")]
NULLS += [(rec_bwd, k) for k in ("x", "gate", "chunks", "dout", "dx", "dg")]
NULLS += [(rec_step, k) for k in ("x", "gate", "state", "out")]
NULLS += [(rotary, k) for k in ("q", "qo", "turns")]
NULLS += [(gn_fwd, k) for k in ("x", "out")] + [(gn_bwd, k) for k in ("x", "dout", "dx")]


@pytest.mark.parametrize("call,name", NULLS, ids=lambda v: getattr(v, "__name__", v))
def test_null_pointers(call, name):
    assert call(**{name: None}) == la.LA_ERR_NULL


def test_pointers_that_go_together():
    assert rotary(k=P) == la.LA_ERR_NULL
    assert rotary(ko=P) == la.LA_ERR_NULL
    assert gn_bwd(gate=P) == la.LA_ERR_NULL
    assert gn_bwd(dgate=P) == la.LA_ERR_NULL


@pytest.mark.parametrize("call", [rec_fwd, rec_bwd, rec_step, rotary, gn_fwd, gn_bwd])
@pytest.mark.parametrize("size", [dict(B=0), dict(H=-1), dict(d=0), dict(d=(1 << 20) + 1),
                                  dict(B=1 << 30, H=1 << 30)])
def test_sizes(call, size):
    assert call(**size) == la.LA_ERR_SHAPE
    if call is not rec_step:
        assert call(L=0) == la.LA_ERR_SHAPE


@pytest.mark.parametrize("call", [rec_fwd, rec_bwd, rec_step])
def test_kinds(call):
    assert call(dtype=2) == la.LA_ERR_UNSUPPORTED
    assert call(gdtype=-1) == la.LA_ERR_UNSUPPORTED
    assert call(kind=3) == la.LA_ERR_UNSUPPORTED


def test_rotary_arguments():
    assert rotary(rot=7) == la.LA_ERR_SHAPE
    assert rotary(rot=10) == la.LA_ERR_SHAPE
    assert rotary(rot=-2) == la.LA_ERR_SHAPE
    assert rotary(k=P, ko=P, Hk=0) == la.LA_ERR_SHAPE
    assert rotary(layout=2) == la.LA_ERR_UNSUPPORTED
    assert rotary(dtype=5) == la.LA_ERR_UNSUPPORTED
    assert rotary(amp=float("nan")) == la.LA_ERR_ARG


def test_group_norm_arguments():
    for call in (gn_fwd, gn_bwd):
        for eps in (0.0, -1.0, float("nan"), float("inf")):
            assert call(eps=eps) == la.LA_ERR_ARG
        assert call(act=2) == la.LA_ERR_UNSUPPORTED
        assert call(d=8193) == la.LA_ERR_UNSUPPORTED
        assert call(dtype=2) == la.LA_ERR_UNSUPPORTED
    need = la.la_group_norm_bwd_workspace_bytes(2, 3, 5, 8)
    assert need > 0
    assert gn_bwd(dw=P) == la.LA_ERR_WORKSPACE
    assert gn_bwd(db=P, ws=P, wsb=need - 1) == la.LA_ERR_WORKSPACE
    assert la.la_group_norm_bwd_workspace_bytes(0, 3, 5, 8) == 0
    assert la.la_group_norm_bwd_workspace_bytes(2, 3, 5, 8193) == 0


# (name of a strides argument, is it an output's)
STRIDES = [(rec_fwd, "sx", 0), (rec_fwd, "sg", 0), (rec_fwd, "so", 1), (rec_bwd, "sx", 0), (rec_bwd, "sdo", 0),
           (rec_bwd, "sdx", 1), (rec_bwd, "sdg", 1), (rotary, "sq", 0), (rotary, "sqo", 1), (gn_fwd, "sx", 0),
           (gn_fwd, "so", 1), (gn_bwd, "sdo", 0), (gn_bwd, "sdx", 1)]


@pytest.mark.parametrize("call,name,output", STRIDES)
def test_strides(call, name, output):
    assert call(**{name: st(-120, 40, 8)}) == la.LA_ERR_ARG
    assert call(**{name: st(1 << 60, 40, 8)}) == la.LA_ERR_ARG
    if output:  # two elements in one place
        assert call(**{name: st(120, 40, 0)}) == la.LA_ERR_ARG
        assert call(**{name: st(120, 40, 7)}) == la.LA_ERR_ARG
        assert call(**{name: st(120, 39, 8)}) == la.LA_ERR_ARG
        assert call(**{name: st(119, 8, 24)}) == la.LA_ERR_ARG


def test_alignment():
    assert rec_fwd(x=ODD) == la.LA_ERR_ARG
    assert rec_fwd(gate=ODD, gdtype=la.LA_BF16) == la.LA_ERR_ARG
    assert rec_fwd(h0=ctypes.c_void_p((1 << 20) + 2)) == la.LA_ERR_ARG
    assert rec_bwd(dx=ODD) == la.LA_ERR_ARG
    assert rec_step(state=ODD) == la.LA_ERR_ARG
    assert rotary(turns=ctypes.c_void_p((1 << 20) + 4)) == la.LA_ERR_ARG
    assert rotary(qo=ODD, dtype=la.LA_BF16) == la.LA_ERR_ARG
    assert gn_fwd(w=ODD) == la.LA_ERR_ARG
    assert gn_bwd(dout=ODD, dtype=la.LA_BF16) == la.LA_ERR_ARG


def test_binding_refuses_lengths_past_32_bits():
    """A length that the C ABI's ints do not hold is refused, not cut to its low 32 bits."""
    torch = pytest.importorskip("torch")
    for axis in range(4):
        shape = [1, 1, 1, 1]
        shape[axis] = (1 << 32) + 1
        x = torch.zeros(1).expand(shape)
        calls = [lambda: la.recurrence_fwd(x, x), lambda: la.recurrence_bwd(x, x, x, x),
                 lambda: la.rotary(x, None, la.RotaryTable(torch.zeros(1, dtype=torch.int64), 2)),
                 lambda: la.group_norm_fwd(x), lambda: la.group_norm_bwd(x, x)]
        if axis:
            calls.append(lambda: la.recurrence_step(x[0], x[0], x[0]))
        for call in calls:
            with pytest.raises(ValueError, match="too long"):
                call()


def test_group_norm_workspace_refusals():
    """A workspace of another device, or one whose elements share memory, is refused."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 1, 1, 8)
    for workspace in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
                      torch.zeros(1 << 16, dtype=torch.uint8, device="meta"),
                      torch.zeros(1 << 16, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace must be contiguous on cpu"):
            la.group_norm_bwd(x, x, weight=torch.ones(8), workspace=workspace)


# ---- the rotary table --------------------------------------------------------------------
def table(rot, base=10000.0, scaling=0, factor=1.0, original=0.0, fast=32.0, slow=1.0):
    out = (ctypes.c_ulonglong * max(1, rot // 2))()
    rc = la.la_rotary_table(rot, base, scaling, factor, original, fast, slow, out)
    return rc, [int(v) for v in out][:max(0, rot // 2)]


@pytest.mark.parametrize("kw", [dict(), dict(base=5e5), dict(scaling=1, factor=8.0),
                                dict(scaling=2, factor=8.0, original=8192.0),
                                dict(scaling=2, factor=32.0, original=2048.0, fast=16.0, slow=2.0)])
@pytest.mark.parametrize("rot", [2, 6, 64, 128])
def test_rotary_table(rot, kw):
    """turns / 2^64 = theta / (2 pi), theta to the roundings of a few 64-bit operations."""
    rc, turns = table(rot, **kw)
    assert rc == la.LA_OK
    names = {0: "none", 1: "linear", 2: "parts"}
    theta = ref.frequencies(rot, kw.get("base", 1e4), names[kw.get("scaling", 0)], kw.get("factor", 1.0),
                            kw.get("original", 0.0), kw.get("fast", 32.0), kw.get("slow", 1.0))
    got = np.array([t / 2.0 ** 64 for t in turns]) * 2 * np.pi
    assert np.all(np.abs(got - theta) <= 16 * 2.0 ** -53 * theta + 2.0 ** -60)


def test_rotary_table_refusals():
    assert table(0)[0] == la.LA_ERR_SHAPE
    assert table(3)[0] == la.LA_ERR_SHAPE
    assert table(4, scaling=3)[0] == la.LA_ERR_UNSUPPORTED
    for kw in (dict(base=0.0), dict(base=float("inf")), dict(scaling=1, factor=0.5),
               dict(scaling=1, factor=float("nan")), dict(scaling=2, factor=2.0, original=0.0),
               dict(scaling=2, factor=2.0, original=8.0, fast=1.0, slow=1.0),
               dict(scaling=2, factor=2.0, original=8.0, slow=0.0), dict(base=1e-300)):
        assert table(64, **kw)[0] == la.LA_ERR_ARG, kw
    assert la.la_rotary_table(4, 1e4, 0, 1.0, 0.0, 32.0, 1.0, None) == la.LA_ERR_NULL


def test_rotary_table_of_many_turns():
    """More turns per position than a double holds with digits to spare are refused; below that
    the fraction of a turn is right to the digits of theta that pow() gives."""
    from fractions import Fraction
    assert table(4, base=1e-34)[0] == la.LA_ERR_ARG  # theta = 1e17: 1.6e16 turns
    assert table(4, base=2.0 ** -106)[0] == la.LA_ERR_ARG  # 2^53 / (2 pi) = 1.4e15 turns, more than 2^50
    rc, turns = table(4, base=2.0 ** -100)  # theta = 2^50, exactly
    assert rc == la.LA_OK
    inv = Fraction(15915494309189533576888376337251436203445964574046, 10 ** 50)  # 1 / (2 pi)
    want = (2 ** 50 * inv) % 1
    # inv_lo has 53 bits behind 2^-56: 2^50 2^-109, and the result is cut to 2^-64
    assert abs(Fraction(turns[1], 2 ** 64) - want) <= Fraction(1, 2 ** 58)


# ---- the 64-bit forms ---------------------------------------------------------------------
def numeric(f, v, h=1e-6):
    """Central differences of a scalar function."""
    out = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + h
        up = f()
        v[i] = keep - h
        down = f()
        v[i] = keep
        out[i] = (up - down) / (2 * h)
    return out


@pytest.mark.parametrize("kind", ["value", "log", "sigmoid"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("lengths", [None, [5, 2]])
def test_recurrence_gradients_by_differences(kind, complement, lengths):
    rng = np.random.default_rng(3)
    shape = (2, 1, 5, 3)
    x, dout = rng.normal(size=shape), rng.normal(size=shape)
    g = {"value": rng.uniform(0.1, 0.9, shape), "log": -rng.uniform(0.1, 2, shape),
         "sigmoid": rng.normal(size=shape)}[kind]
    h0, dlast = rng.normal(size=(2, 1, 3)), rng.normal(size=(2, 1, 3))

    def loss():
        out, last, _ = ref.recurrence(x, g, kind, complement, h0, lengths)
        return (out * dout).sum() + (last * dlast).sum()

    dx, dg, dh0, _ = ref.recurrence_grads(x, g, dout, dlast, kind, complement, h0, lengths)
    for got, v in ((dx, x), (dg, g), (dh0, h0)):
        assert np.allclose(got, numeric(loss, v), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_group_norm_gradients_by_differences(center, gated, act):
    rng = np.random.default_rng(4)
    x = rng.normal(size=(2, 2, 3, 4)) + 0.5
    w, b = rng.normal(size=(2, 4)), rng.normal(size=(2, 4))
    gate = rng.normal(size=(2, 3, 2, 4)) if gated else None
    dout = rng.normal(size=(2, 3, 2, 4))

    def loss():
        return (ref.group_norm(x, w, b, gate, 1e-3, act, center)["out"][0] * dout).sum()

    r = ref.group_norm(x, w, b, gate, 1e-3, act, center, dout)
    assert np.allclose(np.swapaxes(r["dx"][0], 1, 2), numeric(loss, x), rtol=1e-5, atol=1e-6)
    assert np.allclose(r["dw"][0], numeric(loss, w), rtol=1e-5, atol=1e-6)
    assert np.allclose(r["db"][0], numeric(loss, b), rtol=1e-5, atol=1e-6)
    if gated:
        assert np.allclose(r["dgate"][0], numeric(loss, gate), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_is_a_rotation(layout):
    """Norms stay, the inverse undoes it, and q.k depends on the distance alone."""
    rng = np.random.default_rng(5)
    q, k = rng.normal(size=(1, 1, 4, 10)), rng.normal(size=(1, 1, 4, 10))
    theta = ref.frequencies(8)
    p = np.array([[0, 3, 100, 7]])
    a, _ = ref.rotary(q, p, theta, layout)
    assert np.allclose((a * a).sum(-1), (q * q).sum(-1))
    assert np.allclose(ref.rotary(a, p, theta, layout, inverse=True)[0], q)
    b, _ = ref.rotary(k, p + 5, theta, layout)
    a2, _ = ref.rotary(q, p + 1000, theta, layout)
    b2, _ = ref.rotary(k, p + 1005, theta, layout)
    assert np.allclose((a[..., :8] * b[..., :8]).sum(-1), (a2[..., :8] * b2[..., :8]).sum(-1))
