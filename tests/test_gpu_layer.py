"""The operators around the attention (recurrence, rotary positions, group norm) on the GPU
against their 64-bit forms, within the bounds derived there."""
import numpy as np
import pytest

import layer_reference as ref

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


def torch_type(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def dev(v, dtype="f32"):
    """numpy -> CUDA tensor rounded to dtype."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(v)).to(torch_type(dtype)).cuda()


def host(t):
    return t.double().cpu().numpy()


def check(name, got, value, bound, dtype="f32"):
    """|got - value| within the bound, rounding to the stored type included."""
    got = host(got).reshape(value.shape)
    assert np.isfinite(got).all(), name
    off = np.abs(got - value) - ref.stored(bound, value, dtype)
    i = np.unravel_index(np.argmax(off), off.shape)
    assert off[i] <= 0, f"{name}{i}: got {got[i]!r}, is {value[i]!r}, bound {bound[i]!r}"


def strided(t, order):
    """A copy of [B, H, L, d] whose memory is [B, L, H, d + 8] ("blh") or as it is (None)."""
    import torch
    if order is None:
        return t.clone()
    B, H, L, d = t.shape
    rows = torch.full((B, L, H, d + 8), float("nan"), dtype=t.dtype, device=t.device)
    v = rows[..., :d].transpose(1, 2)
    v.copy_(t)
    return v


# ---- recurrence ----------------------------------------------------------------------------
def gate_values(rng, kind, shape, resets=True):
    n = rng.normal(size=shape) * 1.5 + 2.0
    if kind == "sigmoid":
        return n
    g = 1 / (1 + np.exp(-n)) if kind == "value" else -np.log1p(np.exp(-n))
    if resets:
        r = rng.random(shape) < 0.02
        g = np.where(r, 0.0 if kind == "value" else -np.inf, g)
    return g


# (B, H, L, d): one row, seams of the chunks, odd sizes, several column blocks
REC_SHAPES = [(1, 1, 1, 1), (2, 3, 5, 7), (1, 2, 127, 64), (2, 1, 128, 32), (1, 1, 129, 40), (1, 2, 300, 130),
              (3, 2, 1000, 48), (1, 1, 2500, 64), (2, 2, 513, 256), (1, 3, 260, 33),
              (1, 1, 63, 64), (1, 1, 64, 66), (1, 2, 65, 64), (40, 4, 70, 64), (90, 1, 129, 128)]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")]


def run_recurrence(la, shape, kind, complement, dtype, gate_dtype, order=None, lengths=None, initial=True, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    B, H, L, d = shape
    x, g = dev(rng.normal(size=shape), dtype), dev(gate_values(rng, kind, shape), gate_dtype)
    dout = dev(rng.normal(size=shape), dtype)
    h0 = dev(rng.normal(size=(B, H, d))) if initial else None
    dlast = dev(rng.normal(size=(B, H, d))) if initial else None
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    xs, gs, ds = strided(x, order), strided(g, order), strided(dout, order)
    if lengths is not None:  # what stands behind a sequence's end is never read
        for b, k in enumerate(lengths):
            for v in (xs, gs, ds):
                v[b, :, max(0, k):] = float("nan")
    kw = dict(gate_kind=kind, complement=complement, lengths=n)
    out, dx = strided(torch.zeros_like(x), order), strided(torch.zeros_like(x), order)
    dg = strided(torch.zeros_like(g), order)
    out, last, chunks = la.recurrence_fwd(xs, gs, h0=h0, save_chunks=True, out=out, **kw)
    plain = la.recurrence_fwd(xs, gs, h0=h0, **kw)
    assert torch.equal(plain[0], out) and torch.equal(plain[1], last)
    dx, dg, dh0 = la.recurrence_bwd(xs, gs, chunks, ds, dh_last=dlast, dx=dx, dgate=dg, **kw)
    clip = None if lengths is None else [min(max(k, 0), L) for k in lengths]
    hx, hg, hd = host(x), host(g), host(dout)
    hh = None if h0 is None else host(h0)
    hl = None if dlast is None else host(dlast)
    want, wlast, before = ref.recurrence(hx, hg, kind, complement, hh, clip)
    bound = ref.recurrence_bounds(hx, hg, kind, complement, hh, clip)
    on = np.ones((B, 1, L, 1)) if clip is None else (np.arange(L) < np.array(clip)[:, None])[:, None, :, None]
    check("out", out, want, bound * on, dtype)
    check("last", last, wlast, bound[:, :, -1])
    n_c = la.LA_RECURRENCE_CHUNK
    cb = np.concatenate([np.zeros((B, H, 1, d)), bound[:, :, n_c - 1:-1:n_c]], 2)[:, :, :-(-L // n_c)]
    check("chunks", chunks, before[:, :, ::n_c], cb)
    wx, wg, w0, _ = ref.recurrence_grads(hx, hg, hd, hl, kind, complement, hh, clip)
    bx, bg, b0 = ref.recurrence_grad_bounds(hx, hg, hd, hl, kind, complement, hh, clip)
    check("dx", dx, wx, bx * on, dtype)
    check("dg", dg, wg, bg * on, gate_dtype)
    check("dh0", dh0, w0, b0)


@pytest.mark.parametrize("shape", REC_SHAPES, ids=str)
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
def test_recurrence_shapes(la, shape, dtype, gate_dtype):
    run_recurrence(la, shape, "log", True, dtype, gate_dtype)


@pytest.mark.parametrize("kind", ["value", "log", "sigmoid"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_recurrence_gates(la, kind, complement, dtype):
    run_recurrence(la, (2, 2, 400, 64), kind, complement, dtype, dtype, seed=1)


@pytest.mark.parametrize("d", [64, 100, 7])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_recurrence_strided(la, d, dtype):
    run_recurrence(la, (2, 3, 200, d), "sigmoid", True, dtype, "f32", order="blh", seed=2)


@pytest.mark.parametrize("lengths", [[0, 1, 300], [128, 129, 127], [-5, 1000, 256]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 9])
def test_recurrence_padded(la, lengths, dtype, d):
    run_recurrence(la, (3, 2, 300, d), "value", False, dtype, dtype, lengths=lengths, seed=3)
    run_recurrence(la, (3, 2, 300, d), "log", True, dtype, "f32", lengths=lengths, initial=False, seed=4)


def test_recurrence_long(la):
    """A sequence of many chunks and few channels, where it is shared out over time."""
    run_recurrence(la, (1, 1, 20000, 64), "log", False, "f32", "f32", seed=5)


@pytest.mark.parametrize("kind", ["value", "log", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 7), (8, 16, 128)], ids=str)
def test_recurrence_step(la, kind, dtype, shape):
    """Steps give the forward's rows; the state is updated in place."""
    rng = np.random.default_rng(6)
    B, H, d = shape
    L = 6
    x = dev(rng.normal(size=(B, H, L, d)), dtype)
    g = dev(gate_values(rng, kind, (B, H, L, d)), dtype)
    state = dev(rng.normal(size=shape))
    hx, hg, h0 = host(x), host(g), host(state)
    want, last, _ = ref.recurrence(hx, hg, kind, True, h0)
    bound = ref.recurrence_bounds(hx, hg, kind, True, h0)
    for t in range(L):
        out = la.recurrence_step(x[:, :, t].contiguous(), g[:, :, t].contiguous(), state, gate_kind=kind,
                                 complement=True)
        check(f"step {t}", out, want[:, :, t], bound[:, :, t], dtype)
    check("state", state, last, bound[:, :, -1])


@pytest.mark.parametrize("kind,zero", [("value", 0.0), ("log", -np.inf), ("sigmoid", -np.inf)])
@pytest.mark.parametrize("row", [1, 7, 8, 15, 16, 63, 64, 127, 128, 200])
def test_recurrence_gate_zero_forgets_everything(la, kind, zero, row):
    """A gate of 0 starts anew, whatever stood before it: infinities, NaN."""
    rng = np.random.default_rng(7)
    shape = (1, 2, 260, 64)
    x, g = rng.normal(size=shape), gate_values(rng, kind, shape, resets=False)
    g[:, :, row] = zero
    bad = x.copy()
    bad[:, 0, row - 1], bad[:, 1, 0] = np.inf, np.nan
    a, la_last = la.recurrence_fwd(dev(bad), dev(g), gate_kind=kind)
    b, lb_last = la.recurrence_fwd(dev(x[:, :, row:]), dev(g[:, :, row:]), gate_kind=kind)
    check("rows", a[:, :, row:], host(b), 2 * ref.recurrence_bounds(x[:, :, row:], g[:, :, row:], kind, False))
    assert np.isfinite(host(la_last)).all()
    assert not np.isfinite(host(a[:, 0, row - 1])).any()
    # backwards: a gradient of infinity behind the zero gate stays behind it
    _, _, chunks = la.recurrence_fwd(dev(x), dev(g), gate_kind=kind, save_chunks=True)
    do = np.ones(shape)
    do[:, :, row] = np.inf
    dx, _, dh0 = la.recurrence_bwd(dev(x), dev(g), chunks, dev(do), gate_kind=kind)
    assert np.isfinite(host(dx[:, :, :row])).all() and np.isfinite(host(dh0)).all()


def test_recurrence_aliases_and_streams(la):
    """h_last over h0, a stream of one's own, and equal bits from equal calls."""
    import torch
    rng = np.random.default_rng(8)
    shape = (1, 2, 3000, 64)
    x, g, h = dev(rng.normal(size=shape)), dev(gate_values(rng, "log", shape)), dev(rng.normal(size=(1, 2, 64)))
    out, last, chunks = la.recurrence_fwd(x, g, h0=h, gate_kind="log", save_chunks=True)
    side = torch.cuda.Stream()
    state, again = h.clone(), torch.empty_like(out)
    side.wait_stream(torch.cuda.current_stream())
    rc = la.la_recurrence_fwd(x.data_ptr(), g.data_ptr(), state.data_ptr(), None, again.data_ptr(),
                              state.data_ptr(), None, *shape, None, None, None, la.LA_GATE_LOG, 0, la.LA_F32,
                              la.LA_F32, side.cuda_stream)
    assert rc == la.LA_OK
    side.synchronize()
    assert torch.equal(again, out) and torch.equal(state, last)
    do = dev(rng.normal(size=shape))
    first = la.recurrence_bwd(x, g, chunks, do, dh_last=h, gate_kind="log")
    second = la.recurrence_bwd(x, g, chunks, do, dh_last=h, gate_kind="log")
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    grad = h.clone()
    dx, dg = torch.empty_like(x), torch.empty_like(g)
    rc = la.la_recurrence_bwd(x.data_ptr(), g.data_ptr(), chunks.data_ptr(), None, do.data_ptr(), grad.data_ptr(),
                              dx.data_ptr(), dg.data_ptr(), grad.data_ptr(), *shape, None, None, None, None, None,
                              la.LA_GATE_LOG, 0, la.LA_F32, la.LA_F32, torch.cuda.current_stream().cuda_stream)
    assert rc == la.LA_OK
    assert torch.equal(dx, first[0]) and torch.equal(dg, first[1]) and torch.equal(grad, first[2])


@pytest.mark.parametrize("raw", [None, 0, 1, 2])
def test_memory_of_a_named_stream(la, raw):
    """What a call with stream= allocates belongs to that stream: a stream of one's own (None), and
    the handles 0 and 1 (the default stream) and 2 (the thread's)."""
    import torch
    rng = np.random.default_rng(17)
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw is None else raw
    owner = 0 if raw == 1 else handle
    B, H, L, d = 2, 3, 200, 64
    x, g, dout = (dev(rng.normal(size=(B, H, L, d))) for _ in range(3))
    do = dev(rng.normal(size=(B, L, H * d)))
    w = dev(rng.normal(size=H * d))
    table = la.rotary_table(d)
    torch.cuda.synchronize()

    def calls(**on):
        out, last, chunks = la.recurrence_fwd(x, g, save_chunks=True, **on)
        dx, dg, dh0 = la.recurrence_bwd(x, g, chunks, dout, **on)
        step = la.recurrence_step(x[:, :, 0].contiguous(), g[:, :, 0].contiguous(), last.clone(), **on)
        q, k = la.rotary(x, g, table, **on)
        y = la.group_norm_fwd(x, w, **on)
        nx, _, dw, _ = la.group_norm_bwd(x, do, w, **on)
        return out, last, chunks, dx, dg, dh0, step, q, k, y, nx, dw

    want = calls()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.ExternalStream(owner) if owner else torch.cuda.default_stream()):
        got = calls(stream=handle)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = la.group_norm_bwd(x, do, w, stream=handle)[::2] + la.rotary(x, g, table, stream=handle)
    assert torch.cuda.current_stream().cuda_stream == 0
    torch.cuda.synchronize()
    segments = [(s["address"], s["total_size"], s["stream"]) for s in torch.cuda.memory_snapshot()]
    for t in got:
        assert [o for a, n, o in segments if a <= t.data_ptr() < a + n] == [owner]


def test_offsets_past_32_bits(la):
    """Rows 2^31 elements apart, for every operator."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    rng = np.random.default_rng(9)
    L, d, step = 3, 64, (1 << 31) + 64
    big = torch.empty((L - 1) * step + d, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((1, 1, L, d), (0, 0, step, 1))
    res = torch.empty_like(big).as_strided((1, 1, L, d), (0, 0, step, 1))
    x, g = dev(rng.normal(size=(1, 1, L, d)), "bf16"), dev(rng.normal(size=(1, 1, L, d)), "bf16")
    far.copy_(x)
    near, _, chunks = la.recurrence_fwd(x, g, save_chunks=True)
    la.recurrence_fwd(far, g, out=res)
    assert torch.equal(res.contiguous(), near)
    dx, dg, _ = la.recurrence_bwd(x, g, chunks, x)
    la.recurrence_bwd(far, g, chunks, far, dx=res)
    assert torch.equal(res.contiguous(), dx)
    table = la.rotary_table(d)
    q, _ = la.rotary(x, None, table)
    la.rotary(far, None, table, q_out=res)
    assert torch.equal(res.contiguous(), q)
    y = la.group_norm_fwd(x)
    la.group_norm_fwd(far, out=res[:, 0])
    assert torch.equal(res[:, 0].contiguous(), y)
    gx = la.group_norm_bwd(x, y)[0]
    la.group_norm_bwd(far, y, dx=res)
    assert torch.equal(res.contiguous(), gx)


def test_recurrence_without_the_optional_buffers(la):
    """No h0, h_last, chunk states, dh_last, dh0: the rest is the same."""
    import torch
    rng = np.random.default_rng(17)
    shape = (2, 1, 700, 64)
    x, g, do = dev(rng.normal(size=shape), "bf16"), dev(rng.normal(size=shape), "bf16"), dev(rng.normal(size=shape), "bf16")
    want, _, chunks = la.recurrence_fwd(x, g, save_chunks=True)
    out = torch.empty_like(x)
    kinds = (la.LA_GATE_SIGMOID, 0, la.LA_BF16, la.LA_BF16, torch.cuda.current_stream().cuda_stream)
    p = [t.data_ptr() for t in (x, g, out)]
    assert la.la_recurrence_fwd(p[0], p[1], None, None, p[2], None, None, *shape, None, None, None, *kinds) == la.LA_OK
    assert torch.equal(out, want)
    dx, dg, _ = la.recurrence_bwd(x, g, chunks, do)
    rx, rg = torch.empty_like(x), torch.empty_like(g)
    assert la.la_recurrence_bwd(p[0], p[1], chunks.data_ptr(), None, do.data_ptr(), None, rx.data_ptr(), rg.data_ptr(),
                                None, *shape, None, None, None, None, None, *kinds) == la.LA_OK
    assert torch.equal(rx, dx) and torch.equal(rg, dg)


def test_recurrence_stalled_wait_times_out(la, monkeypatch):
    """Blocks of a cluster that hear nothing of one another give up, say so, and leave the context
    as it was."""
    import time

    import torch
    rng = np.random.default_rng(18)
    shape = (1, 1, 2000, 32)
    x, g = dev(rng.normal(size=shape)), dev(rng.normal(size=shape))
    stream = torch.cuda.current_stream().cuda_stream
    want, _, chunks = la.recurrence_fwd(x, g, save_chunks=True)
    dx = la.recurrence_bwd(x, g, chunks, x)[0]
    assert la.la_last_device_status(stream) == la.LA_OK
    monkeypatch.setenv("LA_DEBUG_STALL", "1")
    monkeypatch.setenv("LA_DEBUG_TIMEOUT_NS", "100000000")  # 0.1 s
    for call in (lambda: la.recurrence_fwd(x, g), lambda: la.recurrence_bwd(x, g, chunks, x)):
        t0 = time.time()
        call()
        assert la.la_last_device_status(stream) == la.LA_ERR_TIMEOUT
        assert time.time() - t0 < 20
        assert la.la_last_device_status(stream) == la.LA_OK
    monkeypatch.delenv("LA_DEBUG_STALL")
    monkeypatch.delenv("LA_DEBUG_TIMEOUT_NS")
    assert torch.equal(la.recurrence_fwd(x, g)[0], want) and torch.equal(la.recurrence_bwd(x, g, chunks, x)[0], dx)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_recurrence_stalled_wait_in_a_long_sequence(la, monkeypatch, dtype):
    """The same with steps left after the one whose wait ran out: one wait a block, not one a step."""
    import time

    import torch
    rng = np.random.default_rng(19)
    shape = (1, 1, 30000, 32)
    x, g = dev(rng.normal(size=shape), dtype), dev(rng.normal(size=shape), dtype)
    stream = torch.cuda.current_stream().cuda_stream
    want, _, chunks = la.recurrence_fwd(x, g, save_chunks=True)
    dx = la.recurrence_bwd(x, g, chunks, x)[0]
    assert la.la_last_device_status(stream) == la.LA_OK
    with monkeypatch.context() as m:
        m.setenv("LA_DEBUG_STALL", "1")
        m.setenv("LA_DEBUG_TIMEOUT_NS", "400000000")  # 0.4 s; a wait a step would take 3 s or more
        for call in (lambda: la.recurrence_fwd(x, g), lambda: la.recurrence_bwd(x, g, chunks, x)):
            t0 = time.time()
            call()
            assert la.la_last_device_status(stream) == la.LA_ERR_TIMEOUT
            assert time.time() - t0 < 2
    assert torch.equal(la.recurrence_fwd(x, g)[0], want) and torch.equal(la.recurrence_bwd(x, g, chunks, x)[0], dx)


FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
import torch
import chunkwise_causal_linear_gb300 as la
x = torch.randn(1, 2, 900, 64, device="cuda")
table = la.rotary_table(64)
w = torch.ones(128, device="cuda")
S, _ = la.decode_state(1, 1, 8, 8)  # a call of the library before the capture, none of these operators
q = torch.randn(1, 1, 8, device="cuda")
la.decode_step(q, q, q, S)
torch.cuda.synchronize()
def step():
    h, _, chunks = la.recurrence_fwd(x, x, save_chunks=True)
    y = la.group_norm_fwd(h, w, w)
    dh = la.group_norm_bwd(h, y, w, w)
    return h, y, *dh[2:], *la.recurrence_bwd(x, x, chunks, dh[0]), la.rotary(x, None, table)[0]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(held, step()))
print("captured first")
"""


def test_first_calls_inside_a_capture():
    """The operators' first calls of a process, captured: nothing they set up disturbs the capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


# ---- rotary positions ------------------------------------------------------------------------
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,L,d,rot", [(1, 1, 1, 1, 2, 2), (2, 3, 1, 5, 10, 6), (1, 4, 2, 33, 64, 64),
                                             (2, 2, 2, 7, 128, 32), (1, 5, 5, 20, 80, 80), (3, 1, 1, 9, 7, 4),
                                             (1, 2, 1, 4, 6, 0), (70, 16, 4, 1, 128, 128), (1, 3, 3, 11, 96, 48)])
def test_rotary(la, layout, dtype, B, H, Hk, L, d, rot):
    import torch
    rng = np.random.default_rng(10)
    q, k = dev(rng.normal(size=(B, H, L, d)), dtype), dev(rng.normal(size=(B, Hk, L, d)), dtype)
    pos = rng.integers(0, 1000, size=(B, L)).astype(np.int32)
    table = la.rotary_table(rot) if rot else la.RotaryTable(torch.empty(0, dtype=torch.int64, device="cuda"), 0)
    theta = ref.frequencies(rot)
    for inverse in (False, True):
        for order in (None, "blh"):
            qo, ko = la.rotary(strided(q, order), strided(k, order), table, positions=torch.from_numpy(pos).cuda(),
                               layout=layout, inverse=inverse)
            for got, src in ((qo, q), (ko, k)):
                want, bound = ref.rotary(host(src), pos, theta, layout, inverse)
                check("rotary", got, want, bound, dtype)
                assert torch.equal(got[..., rot:], src[..., rot:])
    # in place, and into strided outputs
    q2, k2 = strided(q, "blh"), k.clone()
    la.rotary(q2, k2, table, positions=torch.from_numpy(pos).cuda(), layout=layout, inverse=True, q_out=q2, k_out=k2)
    assert torch.equal(q2.contiguous(), qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)),
                                        ("parts", dict(factor=8.0, original_length=8192, amplitude=1.2))])
def test_rotary_far_positions(la, scaling, kw):
    """Positions to 2^31 - 1 and below zero; by an offset and by a list."""
    import torch
    rng = np.random.default_rng(11)
    pos = np.array([[0, 1, 2 ** 24 + 1, 2 ** 31 - 1, -1, -123456789, 10 ** 6, 10 ** 9]], dtype=np.int32)
    x = dev(rng.normal(size=(1, 2, 8, 64)))
    table = la.rotary_table(64, scaling=scaling, **kw)
    theta = ref.frequencies(64, 1e4, scaling, kw.get("factor", 1.0), kw.get("original_length", 0.0))
    got, _ = la.rotary(x, None, table, positions=torch.from_numpy(pos).cuda())
    want, bound = ref.rotary(host(x), pos, theta, "half", amplitude=kw.get("amplitude", 1.0))
    check("far", got, want, bound)
    got, none = la.rotary(x, None, table, offset=10 ** 6)
    want, bound = ref.rotary(host(x), 10 ** 6 + np.arange(8)[None], theta, "half", amplitude=kw.get("amplitude", 1.0))
    check("offset", got, want, bound)
    assert none is None


# ---- group norm --------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated,affine,center,act", [(True, True, True, "silu"), (False, True, True, "silu"),
                                                      (False, False, False, "none"), (True, False, False, "silu"),
                                                      (True, True, False, "none"), (False, True, True, "none")])
@pytest.mark.parametrize("B,H,L,d", [(1, 1, 1, 1), (2, 3, 5, 7), (1, 2, 33, 64), (3, 4, 9, 128), (1, 3, 40, 80),
                                     (2, 1, 17, 256), (1, 2, 6, 300), (1, 1, 5, 1000), (1, 2, 3, 2048),
                                     (1, 1, 2, 5000)])
def test_group_norm(la, dtype, gated, affine, center, act, B, H, L, d):
    rng = np.random.default_rng(12)
    x = dev(rng.normal(size=(B, H, L, d)) + 0.3, dtype)
    w, b = (dev(rng.normal(size=H * d)), dev(rng.normal(size=H * d))) if affine else (None, None)
    gate = dev(rng.normal(size=(B, L, H * d)) * 2, dtype) if gated else None
    dout = dev(rng.normal(size=(B, L, H * d)), dtype)
    kw = dict(gate=gate, activation=act, center=center, eps=1e-5)

    def heads(t):
        return None if t is None else host(t).reshape(B, L, H, d)

    def per_head(t):
        return None if t is None else host(t).reshape(H, d)

    r = ref.group_norm(host(x), per_head(w), per_head(b), heads(gate), 1e-5, act, center, heads(dout))
    for order in (None, "blh"):
        xs = strided(x, order)
        check("out", la.group_norm_fwd(xs, w, b, **kw), *r["out"], dtype)
        dx, dgate, dw, db = la.group_norm_bwd(xs, dout, w, b, dx=strided(x, order), **kw)
        check("dx", dx.transpose(1, 2), *r["dx"], dtype)
        if gated:
            check("dgate", dgate, *r["dgate"], dtype)
        else:
            assert dgate is None
        if affine:
            check("dw", dw, *r["dw"])
            check("db", db, *r["db"])
        else:
            assert dw is None and db is None


def test_group_norm_hard_values(la):
    """A constant group (variance 0), a mean far above the spread, a row with infinity."""
    rng = np.random.default_rng(13)
    x = rng.normal(size=(1, 1, 4, 64))
    x[0, 0, 0] = 3.0
    x[0, 0, 1] = 1000.0 + x[0, 0, 1]
    t = dev(x)
    r = ref.group_norm(host(t), None, None, None, 1e-5, "none", True)
    check("out", la.group_norm_fwd(t, activation="none"), *r["out"])
    t[0, 0, 2, 5] = float("inf")
    out = host(la.group_norm_fwd(t, activation="none"))
    assert np.isfinite(out[0, [0, 1, 3]]).all() and np.isnan(out[0, 2]).all()
    # gates of the largest size: SiLU is 0 or the gate itself, never NaN
    x2 = rng.normal(size=(1, 1, 2, 64))
    gate = np.full((1, 2, 64), 3e38)
    gate[:, 1] = -3e38
    out = host(la.group_norm_fwd(dev(x2), gate=dev(gate)))
    assert (out[0, 1] == 0).all() and not np.isnan(out).any()


def test_group_norm_bits_and_many_rows(la):
    """The weight gradients' sums run in an order of their own sizes alone."""
    import torch
    rng = np.random.default_rng(14)
    B, H, L, d = 2, 3, 3001, 64
    x, dout = dev(rng.normal(size=(B, H, L, d)), "bf16"), dev(rng.normal(size=(B, L, H * d)), "bf16")
    w, b = dev(rng.normal(size=H * d)), dev(rng.normal(size=H * d))
    first, second = la.group_norm_bwd(x, dout, w, b), la.group_norm_bwd(x, dout, w, b)
    assert all(torch.equal(p, q) for p, q in zip(first, second) if p is not None)
    r = ref.group_norm(host(x), host(w).reshape(H, d), host(b).reshape(H, d), None, 1e-5, "silu", True,
                       host(dout).reshape(B, L, H, d))
    check("dw", first[2], *r["dw"])
    check("db", first[3], *r["db"])


# ---- together -------------------------------------------------------------------------------------
def test_refusals_of_the_wrappers(la):
    import torch
    x, g = torch.zeros(1, 2, 4, 8, device="cuda"), torch.zeros(1, 2, 4, 8, device="cuda")
    with pytest.raises(ValueError):
        la.recurrence_fwd(x, g[..., :4])
    with pytest.raises(ValueError):  # channels apart
        la.recurrence_fwd(x.transpose(2, 3).contiguous().transpose(2, 3), g)
    with pytest.raises(TypeError):
        la.recurrence_fwd(x.half(), g)
    with pytest.raises(ValueError):
        la.recurrence_fwd(x, g, h0=torch.zeros(1, 2, 7, device="cuda"))
    with pytest.raises(ValueError):
        la.recurrence_fwd(x.cpu(), g.cpu())
    with pytest.raises(la.LAError):  # every row of the output in one place
        la.recurrence_fwd(x, g, out=torch.zeros(1, 2, 1, 8, device="cuda").expand(1, 2, 4, 8))
    with pytest.raises(ValueError):
        la.recurrence_step(x[:, :, 0], g[:, :, 0], torch.zeros(1, 2, 8, device="cuda"))
    table = la.rotary_table(8)
    with pytest.raises(ValueError):
        la.rotary(x, None, table, positions=torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        la.rotary(x, None, table, positions=torch.zeros(1, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(la.LAError):
        la.rotary(x[..., :4].contiguous(), None, table)
    with pytest.raises(ValueError):
        la.group_norm_fwd(x, weight=torch.ones(8, device="cuda"))
    with pytest.raises(la.LAError):
        la.group_norm_fwd(x, eps=0.0)


def retention(la, q, k, v, gate, table, gamma, w, b):
    """Rotated queries and keys, the decayed attention without its normaliser, group norm, gate."""
    qr, kr = la.rotary(q, k, table)
    y = la.decay_fwd(qr, kr, v, gamma)
    return qr, kr, y, la.group_norm_fwd(y, w, b, gate=gate)


def test_retention_layer_runs_together(la):
    """Projection views -> rotary -> Retention decay -> group norm with gate, forward, backward
    and token by token, against the same chain in 64 bits."""
    import torch
    rng = np.random.default_rng(15)
    B, H, L, d, gamma = 2, 2, 40, 16, 0.97
    rows = dev(rng.normal(size=(B, L, 3, H, d)) / 2)
    q, k, v = (rows[:, :, i].transpose(1, 2) for i in range(3))
    v = v.contiguous()
    gate, dout = dev(rng.normal(size=(B, L, H * d))), dev(rng.normal(size=(B, L, H * d)))
    w, b = dev(1 + 0.1 * rng.normal(size=H * d)), dev(0.1 * rng.normal(size=H * d))
    table = la.rotary_table(d)
    qr, kr, y, out = retention(la, q, k, v, gate, table, gamma, w, b)
    # backward: each operator's own
    dy, dgate, dw, db = la.group_norm_bwd(y, dout, w, b, gate=gate)
    dqr, dkr, dv = la.chunked_bwd(qr, kr, v, dy, gamma=gamma)
    drows = torch.zeros_like(rows)
    la.rotary(dqr, dkr, table, inverse=True, q_out=drows[:, :, 0].transpose(1, 2),
              k_out=drows[:, :, 1].transpose(1, 2))
    # the chain in 64 bits, differentiated
    leaves = {n: t.detach().double().cpu().requires_grad_() for n, t in
              dict(q=q, k=k, v=v, gate=gate, w=w, b=b).items()}
    theta = torch.from_numpy(ref.frequencies(d))
    angle = torch.arange(L, dtype=torch.float64)[:, None] * theta
    c, s = torch.cos(angle), torch.sin(angle)

    def turn(x):
        u, z = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((u * c - z * s, u * s + z * c), -1)

    t = torch.arange(L, dtype=torch.float64)
    mask = torch.where(t[:, None] >= t, gamma ** (t[:, None] - t).clamp(min=0), 0.0)
    y64 = (turn(leaves["q"]) @ turn(leaves["k"]).transpose(-1, -2) * mask) @ leaves["v"]
    xc = y64 - y64.mean(-1, keepdim=True)
    xh = xc / torch.sqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
    o64 = xh.transpose(1, 2).reshape(B, L, H * d) * leaves["w"] + leaves["b"]
    o64 = o64 * leaves["gate"] * torch.sigmoid(leaves["gate"])
    grads = dict(zip(leaves, torch.autograd.grad(o64, list(leaves.values()), dout.double().cpu())))

    def close(name, got, want):
        # fp32 chains of a few hundred operations each: 1e-4 of the largest value
        want = want.detach().numpy()
        assert np.abs(host(got) - want).max() <= 1e-4 * np.abs(want).max(), name

    close("out", out, o64)
    for name, got in dict(q=drows[:, :, 0].transpose(1, 2), k=drows[:, :, 1].transpose(1, 2), v=dv, gate=dgate, w=dw,
                          b=db).items():
        close(name, got, grads[name])
    # decoding: one token at a time
    S, _ = la.decode_state(B, H, d, d)
    for i in range(L):
        q1, k1 = la.rotary(q[:, :, i:i + 1], k[:, :, i:i + 1], table, offset=i)
        o1 = la.decay_decode_step(q1[:, :, 0].contiguous(), k1[:, :, 0].contiguous(), v[:, :, i].contiguous(), S, gamma)
        close(f"token {i}", la.group_norm_fwd(o1[:, :, None], w, b, gate=gate[:, i:i + 1]), o64[:, i:i + 1])


def test_recurrent_layer_captured(la):
    """recurrence -> group norm with gate and back, captured into a graph and replayed on new
    inputs, on a stream of its own."""
    import torch
    rng = np.random.default_rng(16)
    B, H, L, d = 2, 3, 1500, 64
    shape = (B, H, L, d)
    x, g, gate = (torch.zeros(s, device="cuda") for s in (shape, shape, (B, L, H * d)))
    dout, w, b = torch.zeros(B, L, H * d, device="cuda"), dev(rng.normal(size=H * d)), dev(rng.normal(size=H * d))

    def step():
        h, _, chunks = la.recurrence_fwd(x, g, complement=True, save_chunks=True)
        out = la.group_norm_fwd(h, w, b, gate=gate)
        dh, dgate, dw, db = la.group_norm_bwd(h, dout, w, b, gate=gate)
        dx, dg, dh0 = la.recurrence_bwd(x, g, chunks, dh, complement=True)
        return out, dgate, dw, db, dx, dg, dh0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (1, 2):
        for t in (x, g, gate, dout):
            t.copy_(dev(np.random.default_rng(seed).normal(size=tuple(t.shape))))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, step()))
