"""The gated attention without a GPU: what its entry points refuse before anything is launched, and the
64-bit form that the GPU tests compare against (its gradients by central differences)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
import gated_reference as ref  # noqa: E402
from chunkwise_causal_linear_gb300 import build as la_build  # noqa: E402

P = ctypes.c_void_p(1 << 20)  # never dereferenced: every call below fails on the host
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    la_build.build()
    return la.lib()


def st(b, h, l):
    return ctypes.byref(la.la_strides(b, h, l))


def fwd(q=P, k=P, v=P, g=P, s0=None, s1=None, slots=None, lengths=None, out=P, B=2, H=4, Hk=2, L=5, dk=8, dv=8,
        n=0, sq=None, sk=None, sv=None, sg=None, so=None, scale=1.0, dtype=la.LA_F32, ws=None, wsb=0, path=0):
    return la.la_gated_fwd(q, k, v, g, s0, s1, slots, lengths, out, B, H, Hk, L, dk, dv, n, sq, sk, sv, sg, so, scale,
                           dtype, ws, wsb, None, path)


def bwd(q=P, k=P, v=P, g=P, s0=None, lengths=None, dout=P, ds=None, dq=P, dk_=P, dv_=P, dg=None, dgh=None, ds0=None,
        B=2, H=4, Hk=2, L=5, dk=8, dv=8, sq=None, sk=None, sv=None, sg=None, so=None, sdq=None, sdk=None, sdv=None,
        scale=1.0, dtype=la.LA_F32, ws=None, wsb=0, path=0):
    return la.la_gated_bwd(q, k, v, g, s0, lengths, dout, ds, dq, dk_, dv_, dg, dgh, ds0, B, H, Hk, L, dk, dv, sq, sk,
                           sv, sg, so, sdq, sdk, sdv, scale, dtype, ws, wsb, None, path)


def step(q=P, k=P, v=P, g=P, s=P, slots=None, out=P, B=2, H=4, Hk=2, dk=8, dv=8, n=0, sq=None, sk=None, sv=None,
         sg=None, scale=1.0, dtype=la.LA_F32):
    return la.la_gated_step(q, k, v, g, s, slots, out, B, H, Hk, dk, dv, n, sq, sk, sv, sg, scale, dtype, None)


NULLS = [(fwd, k) for k in ("q", "k", "v", "g", "out")] + [(step, k) for k in ("q", "k", "v", "g", "s", "out")]
NULLS += [(bwd, k) for k in ("q", "k", "v", "g", "dout", "dq", "dk_", "dv_")]


@pytest.mark.parametrize("call,name", NULLS, ids=lambda v: getattr(v, "__name__", v))
def test_null_pointers(call, name):
    assert call(**{name: None}) == la.LA_ERR_NULL


@pytest.mark.parametrize("call", [fwd, bwd, step])
@pytest.mark.parametrize("size", [dict(B=0), dict(H=-4), dict(Hk=0), dict(Hk=3), dict(Hk=8), dict(dk=0), dict(dv=-1),
                                  dict(B=1 << 14, H=8), dict(B=1 << 30, H=1 << 30)])
def test_sizes(call, size):
    assert call(**size) == la.LA_ERR_SHAPE
    if call is not step:
        assert call(L=0) == la.LA_ERR_SHAPE


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_what_is_not_supported(call):
    assert call(dtype=2) == la.LA_ERR_UNSUPPORTED
    assert call(dk=257) == la.LA_ERR_UNSUPPORTED
    assert call(dv=300) == la.LA_ERR_UNSUPPORTED
    if call is not step:
        assert call(path=3) == la.LA_ERR_UNSUPPORTED
        assert call(path=la.LA_PATH_TC) == la.LA_ERR_UNSUPPORTED  # fp32, 8 channels


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_arguments(call):
    for scale in (float("nan"), float("inf")):
        assert call(scale=scale) == la.LA_ERR_ARG
    for s in ("sq", "sk", "sv", "sg"):
        assert call(**{s: st(-8, 8, 8)}) == la.LA_ERR_ARG
    assert call(g=ODD) == la.LA_ERR_ARG
    assert call(q=ODD) == la.LA_ERR_ARG


def test_outputs_must_not_fold():
    assert fwd(so=st(0, 40, 8)) == la.LA_ERR_ARG
    for s in ("sdq", "sdk", "sdv"):
        assert bwd(**{s: st(160, 40, 4)}) == la.LA_ERR_ARG


def test_pools():
    assert fwd(slots=P, s0=P) == la.LA_ERR_SHAPE  # n_slots
    assert step(slots=P) == la.LA_ERR_SHAPE
    assert step(s=ODD) == la.LA_ERR_ARG
    assert fwd(s0=ODD) == la.LA_ERR_ARG
    assert bwd(ds0=ODD) == la.LA_ERR_ARG


def test_workspace_sizes():
    assert la.la_gated_workspace_bytes(1, 1, 0, 64, 64, la.LA_BF16) == 0
    assert la.la_gated_workspace_bytes(1, 1, 64, 64, 257, la.LA_BF16) == 0
    assert la.la_gated_bwd_workspace_bytes(1, 4, 3, 64, 64, 64, la.LA_BF16) == 0
    assert la.la_gated_bwd_workspace_bytes(1, 1, 1, 64, 64, 64, la.LA_F32) > 0


def test_wrappers_refuse():
    x = torch.zeros(1, 2, 3, 8)
    with pytest.raises(ValueError, match="CUDA tensors are needed"):
        la.gated_fwd(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="axes"):
        la.gated_fwd(x[0], x, x, torch.zeros(2))
    with pytest.raises(TypeError):
        la.gated_fwd(x.double(), x, x, torch.zeros(2))


@pytest.mark.parametrize("kind", ["head", "token"])
def test_reference_gradients(kind):
    """The reference's gradients against central differences of its forward pass."""
    B, H, Hk, L, d, e = 3, 4, 2, 7, 3, 5
    q, k, v, g, s0, lengths, do, ds = ref.draw(B, H, Hk, L, d, e, torch.float32, kind, True, True, seed=4, resets=0.1)
    grads = ref.backward(q, k, v, g, do, 0.6, s0, lengths, ds)
    x = dict(dq=q.double(), dk=k.double(), dv=v.double(), dg=g.double(), dstate0=s0.double())

    def loss(p):
        out, state = ref.forward(p["dq"], p["dk"], p["dv"], p["dg"], 0.6, p["dstate0"], lengths)
        return float((out * do).sum() + (state * ds).sum())

    gen = torch.Generator().manual_seed(1)
    for name, value in x.items():
        for i in torch.randperm(value.numel(), generator=gen)[:12].tolist():
            if not torch.isfinite(value.view(-1)[i]):
                assert grads[name].reshape(-1)[i] == 0
                continue
            side = []
            for h in (1e-5, -1e-5):
                p = {n: t.clone() for n, t in x.items()}
                p[name].view(-1)[i] += h
                side.append(loss(p))
            want = (side[0] - side[1]) / 2e-5
            assert abs(want - float(grads[name].reshape(-1)[i])) < 1e-6 * (1 + abs(want)), (name, i)
