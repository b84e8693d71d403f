"""The gated attention on the GPU against the 64-bit recurrence: forward, gradients, decoding steps."""
import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
import gated_reference as ref  # noqa: E402
from gated_reference import close  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gpu(x):
    return None if x is None else x.cuda()


def steps_of(L, d, e):
    """Roundings on the way of a term: two a row (decay, new pair), one per product and sum of a row."""
    return 6 * (L + d + e)


# B, H, Hk, L, dk, dv
SIZES = [(1, 1, 1, 1, 8, 8), (2, 3, 3, 2, 64, 64), (3, 4, 2, 63, 64, 64), (2, 2, 2, 64, 128, 128), (2, 4, 1, 65, 128, 64),
         (3, 6, 3, 129, 40, 24), (2, 2, 1, 200, 64, 128), (1, 3, 3, 333, 17, 200), (1, 2, 2, 300, 256, 256),
         (1, 2, 1, 1100, 64, 64), (1, 1, 1, 2100, 128, 128), (4, 16, 16, 130, 64, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["head", "token"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward(size, kind, dtype):
    B, H, Hk, L, d, e = size
    for initial, padded in ((False, False), (True, True)):
        q, k, v, g, s0, n, _, _ = ref.draw(*size, dtype, kind, initial, padded, seed=L)
        scale = d ** -0.5
        out, state = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), scale=scale, state0=gpu(s0), lengths=gpu(n))
        wout, wstate = ref.forward(q, k, v, g, scale, s0, n)
        m = ref.magnitudes(q, k, v, g, scale, s0, n)
        close("out", out, wout, m["out"], dtype, steps_of(L, d, e))
        close("state", state, wstate, m["state"], F32, steps_of(L, d, e))
        assert la.la_last_device_status(None) == la.LA_OK


TC_SIZES = [(1, 2, 2, 1, 64, 64), (2, 4, 2, 65, 64, 128), (2, 2, 1, 127, 128, 64), (1, 2, 2, 700, 128, 128),
            (10, 16, 16, 70, 64, 64), (1, 1, 1, 3000, 64, 128)]


@pytest.mark.parametrize("size", TC_SIZES, ids=lambda s: "x".join(map(str, s)))
def test_paths(size):
    """Both paths named: few heads (cut into segments) and many, each pair of widths."""
    B, H, Hk, L, d, e = size
    q, k, v, g, s0, n, do, ds = ref.draw(*size, BF16, "token", True, True, seed=20)
    want, wstate = ref.forward(q, k, v, g, 0.1, s0, n)
    small = L * d * e * B * H <= 40e6
    m = ref.magnitudes(q, k, v, g, 0.1, s0, n, *((do, ds) if small else ()))
    grads = ref.backward(q, k, v, g, do, 0.1, s0, n, ds) if small else None
    for path in (la.LA_PATH_TC, la.LA_PATH_SIMT):
        out, state = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), scale=0.1, state0=gpu(s0), lengths=gpu(n), path=path)
        close("out", out, want, m["out"], BF16, steps_of(L, d, e))
        close("state", state, wstate, m["state"], F32, steps_of(L, d, e))
        if small:
            check_grads(grads_of(q, k, v, g, do, 0.1, s0, n, ds, path=path), grads, m, BF16, g, steps_of(L, d, e))
        assert la.la_last_device_status(None) == la.LA_OK


def test_the_tensor_cores_refuse():
    """LA_PATH_TC is refused where it does not apply: type, widths, alignment, broadcast."""
    q, k, v, g, _, _, do, _ = ref.draw(1, 2, 2, 40, 64, 64, BF16)
    q, k, v, g, do = (gpu(x) for x in (q, k, v, g, do))
    odd = torch.zeros(1, 2, 40, 65, dtype=BF16, device="cuda")[..., 1:]
    one = k[:, :1].expand(1, 2, 40, 64)
    for a in ((q.float(), k.float(), v.float()), (q[..., :40], k[..., :40], v), (odd, k, v), (q, one, v)):
        with pytest.raises(la.LAError) as e:
            la.gated_fwd(*a, g, path=la.LA_PATH_TC)
        assert e.value.status == la.LA_ERR_UNSUPPORTED
        with pytest.raises(la.LAError) as e:
            la.gated_bwd(*a, g, do.to(a[0].dtype), path=la.LA_PATH_TC)
        assert e.value.status == la.LA_ERR_UNSUPPORTED


def grads_of(q, k, v, g, do, scale, s0, n, ds, **kw):
    names = ("dq", "dk", "dv", "dg", "dstate0")
    return dict(zip(names, la.gated_bwd(gpu(q), gpu(k), gpu(v), gpu(g), gpu(do), scale=scale, state0=gpu(s0),
                                        lengths=gpu(n), dstate=gpu(ds), **kw)))


def check_grads(got, want, m, dtype, g, steps):
    for name in ("dq", "dk", "dv"):
        close(name, got[name], want[name], m[name], dtype, steps)
    close("dstate0", got["dstate0"], want["dstate0"], m["dstate0"], F32, steps)
    # With F_t the gradient of row t's log decay, R_t and C_t the sums of its pairs with earlier rows and with later
    # ones: F_t = F_{t+1} + R_t - C_t from a segment's end on, where F is <dstate, state>. R_t and C_t are parts of the
    # sums of terms' magnitudes of F_t and F_{t+1}, so what the sum to row t has gathered are roundings of its own
    # magnitude and of those of the rows behind it, the end's product among them.
    size = m["dg"]
    if g.dim() == 3:
        size = size + size.mean(-1, keepdim=True) + m["end"][..., None]
    else:
        size = size + m["end"].sum(0)
    close("dg", got["dg"], want["dg"], size, F32, steps)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["head", "token"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_backward(size, kind, dtype):
    B, H, Hk, L, d, e = size
    if L * d * e * B * H > 40e6:
        pytest.skip("the 64-bit states of every row take too much memory")
    for initial, padded in ((False, False), (True, True)):
        q, k, v, g, s0, n, do, ds = ref.draw(*size, dtype, kind, initial, padded, seed=L + 1)
        ds = ds if initial else None
        scale = d ** -0.5
        got = grads_of(q, k, v, g, do, scale, s0, n, ds)
        want = ref.backward(q, k, v, g, do, scale, s0, n, ds)
        m = ref.magnitudes(q, k, v, g, scale, s0, n, do, ds)
        check_grads(got, want, m, dtype, g, steps_of(L, d, e))
        assert la.la_last_device_status(None) == la.LA_OK


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_without_the_decays_gradient(dtype):
    q, k, v, g, s0, n, do, ds = ref.draw(2, 4, 2, 150, 64, 64, dtype, "token", True, True, seed=3)
    a, b = grads_of(q, k, v, g, do, 0.2, s0, n, ds), grads_of(q, k, v, g, do, 0.2, s0, n, ds, decay_grad=False)
    assert b["dg"] is None
    if dtype == F32:
        for name in ("dq", "dk", "dv", "dstate0"):
            assert torch.equal(a[name], b[name])
        return
    # the tensor cores read one bf16 part of the state where no decay's gradient needs three
    want = ref.backward(q, k, v, g, do, 0.2, s0, n, ds)
    m = ref.magnitudes(q, k, v, g, 0.2, s0, n, do, ds)
    check_grads(b | dict(dg=a["dg"]), want, m, dtype, g, steps_of(150, 64, 64))


def step_inputs(q, k, v, g, t):
    gt = g if g.dim() == 1 else g[:, :, t]
    return gpu(q)[:, :, t], gpu(k)[:, :, t], gpu(v)[:, :, t], gpu(gt)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 4, 2, 70, 64, 64), (3, 2, 2, 9, 128, 128), (1, 3, 1, 20, 40, 24), (2, 2, 2, 5, 33, 17),
                                  (1, 2, 2, 4, 256, 256), (1, 1, 1, 3, 1, 1)], ids=lambda s: "x".join(map(str, s)))
def test_steps(size, dtype):
    """Steps of views give the rows of the sequence, and the state behind it."""
    B, H, Hk, L, d, e = size
    for kind in ("head", "token"):
        q, k, v, g, s0, _, _, _ = ref.draw(*size, dtype, kind, True, seed=d)
        scale = d ** -0.5
        want, wstate = ref.forward(q, k, v, g, scale, s0)
        m = ref.magnitudes(q, k, v, g, scale, s0, None)
        state = gpu(s0).clone()
        rows = torch.stack([la.gated_step(*step_inputs(q, k, v, g, t), state, scale=scale) for t in range(L)], 2)
        # no operand is rounded: fp32 but for the output
        half = ref.HALF[dtype]
        err = (rows.double().cpu() - want).abs()
        assert not (err > steps_of(L, d, e) * ref.U * m["out"] + half * want.abs()).any()
        close("state", state, wstate, m["state"], F32, steps_of(L, d, e))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_prompt_then_steps_in_a_pool(dtype):
    """Padded prompts into slots of a pool, continued by a second part of the prompts, then decoded: the
    rows of the whole sequences; the pool's other entries keep their values."""
    B, H, Hk, L, d, e, cut, n = 3, 4, 2, 150, 64, 64, 90, 6
    q, k, v, g, _, _, _, _ = ref.draw(B, H, Hk, L, d, e, dtype, seed=8)
    want, wstate = ref.forward(q, k, v, g, 0.125)
    m = ref.magnitudes(q, k, v, g, 0.125, None, None)
    pool = torch.randn(n, H, d, e, device="cuda")
    before, slots = pool.clone(), torch.tensor([4, 0, 3], dtype=torch.int32, device="cuda")
    dev = [gpu(x) for x in (q, k, v, g)]
    part = lambda i, j: [x[:, :, i:j] for x in dev]  # noqa: E731
    o1, p = la.gated_fwd(*part(0, cut), scale=0.125, slots=slots, state=pool)
    assert p is pool
    o2, _ = la.gated_fwd(*part(cut, L - 8), scale=0.125, slots=slots, state0=pool, state=pool)
    rows = [la.gated_step(*[x[:, :, t] for x in dev], pool, scale=0.125, slots=slots) for t in range(L - 8, L)]
    out = torch.cat((o1, o2, torch.stack(rows, 2)), 2)
    close("out", out, want, m["out"], dtype, steps_of(L, d, e))
    close("state", pool[slots.long()], wstate, m["state"], F32, steps_of(L, d, e))
    rest = [i for i in range(n) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_slots_that_are_none():
    """A negative slot starts from zero and is not kept; one past the pool too, and it is reported."""
    B, H, L, d = 3, 2, 40, 64
    q, k, v, g, _, _, _, _ = ref.draw(B, H, H, L, d, d, F32, seed=9)
    for bad, status in ((-1, la.LA_OK), (5, la.LA_ERR_DEVICE)):
        slots = torch.tensor([1, bad, 0], dtype=torch.int32, device="cuda")
        pool = torch.randn(5, H, d, d, device="cuda")
        first = pool.clone().cpu()
        s0 = torch.stack((first[1], torch.zeros(H, d, d), first[0]))
        want, wstate = ref.forward(q, k, v, g, 1.0, s0)
        m = ref.magnitudes(q, k, v, g, 1.0, s0, None)
        out, _ = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), slots=slots, state0=pool, state=pool)
        close("out", out, want, m["out"], F32, steps_of(L, d, d))
        close("state", pool[[1, 0]], wstate[[0, 2]], m["state"][[0, 2]], F32, steps_of(L, d, d))
        assert torch.equal(pool[2:].cpu(), first[2:])
        assert la.la_last_device_status(None) == status
        pool.copy_(first)
        out = la.gated_step(*step_inputs(q, k, v, g, 0), pool, slots=slots)
        close("step", out, want[:, :, 0], m["out"][:, :, 0], F32, steps_of(1, d, d))
        assert torch.equal(pool[2:].cpu(), first[2:])
        assert la.la_last_device_status(None) == status


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rows_behind_the_end_may_hold_anything(dtype):
    """NaN and infinities behind a sequence's end reach nothing, forwards and backwards."""
    for size in ((3, 2, 1, 100, 64, 64), (2, 3, 3, 150, 128, 128), (2, 2, 2, 70, 24, 40)):
        B, H, Hk, L, d, e = size
        q, k, v, g, s0, n, do, ds = ref.draw(*size, dtype, "token", True, True, seed=11)
        n[0] = L - 37
        clean = grads_of(q, k, v, g, do, 0.3, s0, n, ds)
        out, state = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), scale=0.3, state0=gpu(s0), lengths=gpu(n))
        for b in range(B):
            for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (g, float("nan")), (do, float("-inf"))):
                x[b, :, int(n[b]):] = bad
        got = grads_of(q, k, v, g, do, 0.3, s0, n, ds)
        out2, state2 = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), scale=0.3, state0=gpu(s0), lengths=gpu(n))
        assert torch.equal(out, out2) and torch.equal(state, state2)
        for name in clean:
            assert torch.equal(clean[name], got[name]), name
        for b in range(B):
            assert not out[b, :, int(n[b]):].any()
            assert not any(got[x][b, :, int(n[b]):].any() for x in ("dq", "dk", "dv", "dg"))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_strided_views(dtype):
    """q, k, v, dout and the gradients as views of fused rows, an output into rows of its own."""
    B, H, Hk, L, d, e = 2, 4, 2, 140, 64, 64
    q, k, v, g, s0, n, do, ds = ref.draw(B, H, Hk, L, d, e, dtype, "token", True, True, seed=12)
    rows = torch.zeros(B, L, (H * d + Hk * d + Hk * e), dtype=dtype, device="cuda")
    split = [x.unflatten(-1, (c, -1)).transpose(1, 2)
             for x, c in zip(rows.split([H * d, Hk * d, Hk * e], -1), (H, Hk, Hk))]
    for x, y in zip(split, (q, k, v)):
        x.copy_(y)
    gs = gpu(g).transpose(1, 2).contiguous().transpose(1, 2)
    place = torch.full((B, L, H, e), 7.0, dtype=dtype, device="cuda").transpose(1, 2)
    a, sa = la.gated_fwd(*split, gs, scale=0.1, state0=gpu(s0), lengths=gpu(n), out=place)
    b, sb = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), scale=0.1, state0=gpu(s0), lengths=gpu(n))
    assert a.data_ptr() == place.data_ptr() and torch.equal(a, b) and torch.equal(sa, sb)
    grad = torch.full_like(rows, 7.0)
    dq, dk, dv = (x.unflatten(-1, (c, -1)).transpose(1, 2)
                  for x, c in zip(grad.split([H * d, Hk * d, Hk * e], -1), (H, Hk, Hk)))
    dos = gpu(do).transpose(1, 2).contiguous().transpose(1, 2)
    got = la.gated_bwd(*split, gs, dos, scale=0.1, state0=gpu(s0), lengths=gpu(n), dstate=gpu(ds), dq=dq, dk=dk, dv=dv)
    want = grads_of(q, k, v, g, do, 0.1, s0, n, ds)
    for x, y in zip(got, want.values()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_odd_alignment_and_broadcast(dtype):
    """Rows that do not begin on 16 bytes, and one key head's rows for the whole batch (stride 0)."""
    B, H, L, d = 2, 3, 90, 64
    q, k, v, g, _, _, do, _ = ref.draw(B, H, H, L, d, d, dtype, seed=13)
    k = k[:1].expand(B, H, L, d)
    wide = [torch.zeros(B, H, L, d + 1, dtype=dtype, device="cuda")[..., 1:] for _ in range(2)]
    wide[0].copy_(q)
    wide[1].copy_(v)
    kk = gpu(k[:1]).expand(B, H, L, d)
    out, state = la.gated_fwd(wide[0], kk, wide[1], gpu(g))
    want, wstate = ref.forward(q, k, v, g, 1.0)
    m = ref.magnitudes(q, k, v, g, 1.0, None, None, do)
    close("out", out, want, m["out"], dtype, steps_of(L, d, d))
    close("state", state, wstate, m["state"], F32, steps_of(L, d, d))
    got = dict(zip(("dq", "dk", "dv", "dg", "dstate0"), la.gated_bwd(wide[0], kk, wide[1], gpu(g), gpu(do))))
    check_grads(got, ref.backward(q, k, v, g, do, 1.0), m, dtype, g, steps_of(L, d, d))


@pytest.mark.parametrize("dtype,d", [(F32, 40), (BF16, 64)], ids=["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 300])
def test_the_first_decay_without_a_state(L, dtype, d):
    """Nothing is before the first row: its decay's gradient is 0 itself, not a difference's rounding."""
    q, k, v, g, _, _, do, ds = (gpu(x) for x in ref.draw(3, 4, 2, L, d, d, dtype, seed=L))
    dg = la.gated_bwd(q, k, v, g, do, dstate=ds)[3]
    assert not dg[:, :, 0].any() and (L == 1 or dg[:, :, 1].any())
    if L == 1:
        assert not la.gated_bwd(q, k, v, -torch.rand(4, device="cuda"), do, dstate=ds)[3].any()


def test_a_decay_of_zero_forgets():
    """-inf at every row: each row sees its own pair only, and the decays have no gradient."""
    B, H, L, d = 1, 2, 70, 64
    for dtype in (F32, BF16):
        q, k, v, g, s0, _, do, ds = ref.draw(B, H, H, L, d, d, dtype, "token", True, seed=14, resets=1.1)
        assert torch.isneginf(g).all()
        out, state = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), state0=gpu(s0))
        want, wstate = ref.forward(q, k, v, g, 1.0, s0)
        m = ref.magnitudes(q, k, v, g, 1.0, s0, None, do, ds)
        close("out", out, want, m["out"], dtype, steps_of(1, d, d))
        close("state", state, wstate, m["state"], F32, steps_of(1, d, d))
        got = grads_of(q, k, v, g, do, 1.0, s0, None, ds)
        assert not got["dg"].any() and not got["dstate0"].any()
        check_grads(got, ref.backward(q, k, v, g, do, 1.0, s0, None, ds), m, dtype, g, steps_of(1, d, d))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rate", [0.0, -0.3, -2.0, -30.0, -103.0, -200.0])
def test_segments_of_any_decay(rate, dtype):
    """A long sequence of one head, cut into segments, from no decay to decays that leave nothing of a row's
    neighbour; some rows without, some positive: the rows far from a segment's end are left out of its sum only
    where their decay is below fp32's range."""
    B, H, L, d = 1, 1, 1500, 64
    q, k, v, _, s0, _, do, ds = ref.draw(B, H, H, L, d, d, dtype, "token", True, seed=21)
    gen = torch.Generator().manual_seed(22)
    g = rate * (0.5 + torch.rand(B, H, L, generator=gen))
    for some, value in ((0.0, 0.0), (0.05, 0.0), (0.01, 0.2)):
        gs = torch.where(torch.rand(B, H, L, generator=gen) < some, torch.tensor(value), g)
        want, wstate = ref.forward(q, k, v, gs, 0.1, s0)
        m = ref.magnitudes(q, k, v, gs, 0.1, s0, None, do, ds)
        out, state = la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(gs), scale=0.1, state0=gpu(s0))
        close("out", out, want, m["out"], dtype, steps_of(L, d, d))
        close("state", state, wstate, m["state"], F32, steps_of(L, d, d))
        check_grads(grads_of(q, k, v, gs, do, 0.1, s0, None, ds), ref.backward(q, k, v, gs, do, 0.1, s0, None, ds), m, dtype,
                    gs, steps_of(L, d, d))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 2, 2, 5000, 64, 64), (8, 20, 20, 100, 128, 128)], ids=["few", "many"])
def test_equal_calls_give_equal_bits(size, dtype):
    q, k, v, g, s0, n, do, ds = ref.draw(*size, dtype, "token", True, True, seed=15)
    a, b = (la.gated_fwd(gpu(q), gpu(k), gpu(v), gpu(g), state0=gpu(s0), lengths=gpu(n)) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = (grads_of(q, k, v, g, do, 1.0, s0, n, ds) for _ in range(2))
    assert all(torch.equal(a[x], b[x]) for x in a)


def test_captured_and_on_another_stream():
    """A prompt, its gradients and steps captured into a graph and replayed on new inputs, and called
    on a named stream."""
    size = (2, 4, 2, 200, 64, 64)
    first = [gpu(x) for x in ref.draw(*size, BF16, "token", True, True, seed=16)]
    second = [gpu(x) for x in ref.draw(*size, BF16, "token", True, True, seed=17)]
    held = [x.clone() for x in first]
    pool = held[4].clone()

    def call(stream=None):
        q, k, v, g, s0, n, do, ds = held
        out, state = la.gated_fwd(q, k, v, g, state0=s0, lengths=n, stream=stream)
        grads = la.gated_bwd(q, k, v, g, do, state0=s0, lengths=n, dstate=ds, stream=stream)
        pool.copy_(s0)
        row = la.gated_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g[:, :, 0], pool, stream=stream)
        return [out, state, *grads, row, pool]

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        call()
    warm.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for inputs in (second, first):
        for x, y in zip(held, inputs):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for x, y in zip(got, call()):
            assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        named = call(side.cuda_stream)
    side.synchronize()
    for x, y in zip(named, got):
        assert torch.equal(x, y)


def test_two_calls_at_once():
    """Calls on two streams whose kernels overlap, each with a workspace of its own."""
    sizes = [(1, 3, 3, 3000, 64, 64), (2, 4, 2, 900, 128, 128)]
    ins = [[gpu(x) for x in ref.draw(*size, BF16, "token", True, True, seed=23 + i)] for i, size in enumerate(sizes)]

    def call(i):
        q, k, v, g, s0, n, do, ds = ins[i]
        return [*la.gated_fwd(q, k, v, g, state0=s0, lengths=n), *la.gated_bwd(q, k, v, g, do, state0=s0, lengths=n, dstate=ds)]

    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = call(i)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert la.la_last_device_status(None) == la.LA_OK


FIRST = """
import torch, chunkwise_causal_linear_gb300 as la
torch.manual_seed(0)
q, k, v = (torch.randn(1, 2, 700, 64, device="cuda", dtype=torch.bfloat16) for _ in range(3))
g = -torch.rand(1, 2, 700, device="cuda")
y = torch.randn(3, 5, 256, device="cuda")
pool = torch.zeros(1, 2, 64, 64, device="cuda")
x = torch.randn(1, 1, 8, device="cuda")
la.decode_step(x, x, x, la.decode_state(1, 1, 8, 8)[0])  # the library's first call, none of these operators
torch.cuda.synchronize()
def call():
    a = list(la.gated_fwd(q, k, v, g)) + list(la.gated_bwd(q, k, v, g, v))
    b = list(la.block_norm_fwd(y, y)) + [x for x in la.block_norm_bwd(y, y, y, y).values() if x is not None]
    pool.zero_()
    return a + b + [la.gated_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g[:, :, 0], pool)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = call()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, call()))
"""


def test_first_calls_in_a_capture():
    """A process whose first calls of these operators are captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_a_layer_of_it():
    """As a mixer uses it: rotary positions, gated attention, group norm with a gate; prompts and their
    gradients against the 64-bit forms."""
    B, H, L, d = 2, 3, 130, 64
    q, k, v, g, _, _, do, _ = ref.draw(B, H, H, L, d, d, F32, "head", seed=18)
    gate = torch.randn(B, L, H * d, generator=torch.Generator().manual_seed(2))
    table = la.rotary_table(d)
    qr, kr = la.rotary(gpu(q), gpu(k), table)
    y, _ = la.gated_fwd(qr, kr, gpu(v), gpu(g), scale=d ** -0.5)
    out = la.group_norm_fwd(y, gate=gpu(gate), center=False)
    theta = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    unit = torch.polar(torch.ones(L, d // 2, dtype=torch.float64), torch.arange(L)[:, None] * theta)

    def turn(x):
        z = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double()) * unit
        return torch.cat((z.real, z.imag), -1)

    qt, kt = turn(q), turn(k)
    wy, _ = ref.forward(qt, kt, v, g, d ** -0.5)
    wy = wy / (wy.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    gd = gate.double()
    want = wy.transpose(1, 2).reshape(B, L, H * d) * gd * torch.sigmoid(gd)
    # fp32 through three operators: the attention's steps on the norm's scale
    err = (out.double().cpu() - want).abs().max()
    assert err < steps_of(L, d, d) * ref.U * float(want.abs().max()) * 4
    gy = la.group_norm_bwd(y, gpu(torch.randn(B, L, H * d, generator=torch.Generator().manual_seed(3))), gate=gpu(gate),
                           center=False)[0]
    dq, dk, dv, dg, _ = la.gated_bwd(qr, kr, gpu(v), gpu(g), gy, scale=d ** -0.5)
    w = ref.backward(qr.cpu(), kr.cpu(), v, g, gy.cpu(), d ** -0.5)
    m = ref.magnitudes(qr.cpu(), kr.cpu(), v, g, d ** -0.5, None, None, gy.cpu(), None)
    check_grads(dict(dq=dq, dk=dk, dv=dv, dg=dg, dstate0=torch.zeros(B, H, d, d)), w | dict(dstate0=torch.zeros(B, H, d, d)),
                m | dict(dstate0=torch.ones(B, H, d, d)), F32, g, steps_of(L, d, d))
    back = la.rotary(dq, dk, table, inverse=True)
    assert all(torch.isfinite(x).all() for x in back)
    # and the norms around the layer
    res = gpu(torch.randn(B, L, H * d, generator=torch.Generator().manual_seed(5)))
    h, n = la.block_norm_fwd(out, res, post_norm="none", pre_norm="rms")
    wh = res.double().cpu() + out.double().cpu()
    assert (h.double().cpu() - wh).abs().max() <= 2 * ref.U * float(wh.abs().max())
    wn = wh / (wh.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    assert (n.double().cpu() - wn).abs().max() <= 64 * ref.U * float(wn.abs().max())
    got = la.block_norm_bwd(out, res, None, res, post_norm="none", pre_norm="rms")
    assert torch.equal(got["dy"], got["dr"])
