"""A log decay of -inf between two rows: an infinity or NaN in one of them, or in a first state, does not reach the
other where the -inf lies in another chunk of 64 than the bad row (any other row, on the fp32 path).  Every
value that it must not reach is that of the same call without it, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
import gated_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("dq", "dk", "dv", "dg", "dstate0")
PATHS = [(F32, la.LA_PATH_SIMT), (BF16, la.LA_PATH_SIMT), (BF16, la.LA_PATH_TC)]
IDS = ["f32", "bf16-simt", "bf16-tc"]
# one segment of four chunks, several, and many heads; every pair of widths of the tensor cores
SIZES = [(2, 4, 2, 250, 64, 64), (1, 2, 2, 1100, 128, 128), (10, 16, 16, 200, 64, 128), (1, 3, 1, 700, 128, 64)]
BAD = [float("nan"), float("inf"), float("-inf")]


def inputs(size, dtype):
    q, k, v, g, s0, _, do, ds = (x if x is None else x.cuda() for x in ref.draw(*size, dtype, "token", True, seed=31, resets=0))
    return dict(q=q, k=k, v=v, g=g, s0=s0, do=do, ds=ds)


def forward(x, path):
    return la.gated_fwd(x["q"], x["k"], x["v"], x["g"], scale=0.3, state0=x["s0"], path=path)


def backward(x, path, **kw):
    return dict(zip(NAMES, la.gated_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=0.3, state0=x["s0"], dstate=x["ds"],
                                        path=path, **kw)))


def spoilt(x, at, value, names):
    """A copy of the inputs with row `at` of the first sequence (all heads) spoilt: some channels of it."""
    y = {n: t.clone() for n, t in x.items()}
    for n in names:
        y[n][0, :, at, ::7] = value
    return y


@pytest.mark.parametrize("dtype,path", PATHS, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("cut", [0, 1, 37, 63])
def test_a_reset_forgets_the_first_state(cut, size, dtype, path):
    """A pool's slot that holds anything, and a sequence that begins with -inf or has one within its first chunk."""
    x = inputs(size, dtype)
    x["g"][:, :, cut] = float("-inf")
    out, state = forward(x, path)
    grads = backward(x, path)
    for value in BAD:
        y = x | dict(s0=torch.full_like(x["s0"], value))
        o, s = forward(y, path)
        assert torch.equal(o[:, :, cut:], out[:, :, cut:]) and torch.equal(s, state), value
        got = backward(y, path)
        for name in ("dq", "dk", "dv"):
            assert torch.equal(got[name][:, :, cut:], grads[name][:, :, cut:]), (name, value)
        assert torch.equal(got["dstate0"], grads["dstate0"]), value
    if cut == 0:  # as the step does
        pool = torch.full_like(x["s0"], float("nan"))
        row = la.gated_step(x["q"][:, :, 0], x["k"][:, :, 0], x["v"][:, :, 0], x["g"][:, :, 0], pool, scale=0.3)
        assert torch.isfinite(row).all() and torch.isfinite(pool).all()


@pytest.mark.parametrize("dtype,path", PATHS, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_bad_row_of_an_earlier_document(size, dtype, path):
    x = inputs(size, dtype)
    for bad, cut in ((5, 64), (63, 64 + 20), (40, 127), (5, 130), (100, size[3] - 3)):
        x2 = {n: t.clone() for n, t in x.items()}
        x2["g"][:, :, cut] = float("-inf")
        out, state = forward(x2, path)
        grads = backward(x2, path)
        for value in BAD:
            y = spoilt(x2, bad, value, ("q", "k", "v", "do"))
            o, s = forward(y, path)
            assert torch.equal(o[:, :, cut:], out[:, :, cut:]) and torch.equal(s, state), (bad, cut, value)
            assert torch.equal(o[1:], out[1:])
            for kw in ({}, dict(decay_grad=False)):
                want, got = (grads, backward(y, path)) if not kw else (backward(x2, path, **kw), backward(y, path, **kw))
                for name in ("dq", "dk", "dv"):
                    assert torch.equal(got[name][:, :, cut:], want[name][:, :, cut:]), (name, bad, cut, value)


@pytest.mark.parametrize("dtype,path", PATHS, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_bad_row_of_a_later_document(size, dtype, path):
    """From the end on: the gradients of k and v, and the first state's, of the documents before."""
    x = inputs(size, dtype)
    L = size[3]
    for cut, bad in ((64, 128), (20, 64), (100, 190), (63, L - 1)):
        x2 = {n: t.clone() for n, t in x.items()}
        x2["g"][:, :, cut] = float("-inf")
        for kw in ({}, dict(decay_grad=False)):
            want = backward(x2, path, **kw)
            for value in BAD:
                got = backward(spoilt(x2, bad, value, ("q", "k", "v", "do")), path, **kw)
                for name in ("dq", "dk", "dv"):
                    assert torch.equal(got[name][:, :, :cut], want[name][:, :, :cut]), (name, cut, bad, value)
                assert torch.equal(got["dstate0"], want["dstate0"]), (cut, bad, value)


@pytest.mark.parametrize("dtype,path", PATHS, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_bad_gradient_of_the_last_state(size, dtype, path):
    x = inputs(size, dtype)
    cut = size[3] - 2
    x["g"][:, :, cut] = float("-inf")
    want = backward(x, path)
    for value in BAD:
        got = backward(x | dict(ds=torch.full_like(x["ds"], value)), path)
        for name in ("dq", "dk", "dv"):
            assert torch.equal(got[name][:, :, :cut], want[name][:, :, :cut]), (name, value)
        assert torch.equal(got["dstate0"], want["dstate0"]), value


@pytest.mark.parametrize("dtype,path", PATHS, ids=IDS)
def test_a_bad_row_reaches_its_own_document(dtype, path):
    """Nothing is lost either: without a reset every row behind it is reached."""
    x = inputs((1, 2, 2, 300, 64, 64), dtype)
    y = {n: t.clone() for n, t in x.items()}
    y["k"][0, :, 70] = float("nan")
    out, state = forward(y, path)
    assert torch.isnan(out[:, :, 70:]).all() and torch.isnan(state).all()
    out, _ = forward(x | dict(s0=torch.full_like(x["s0"], float("nan"))), path)
    assert torch.isnan(out).all()
    y = {n: t.clone() for n, t in x.items()}
    y["g"][0, :, 70] = float("nan")
    assert torch.isnan(forward(y, path)[0][:, :, 70:]).all()
