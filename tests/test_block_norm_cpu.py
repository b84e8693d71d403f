"""The norms around a block without a GPU: what their entry points refuse before anything is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
from chunkwise_causal_linear_gb300 import build as la_build  # noqa: E402

P = ctypes.c_void_p(1 << 20)  # never dereferenced: every call below fails on the host
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    la_build.build()
    return la.lib()


def st(b, l):
    return ctypes.byref(la.la_strides(b, 0, l))


def fwd(y=P, r=P, gate=None, w1=None, b1=None, w2=None, b2=None, h=P, n=P, B=2, L=3, d=8, sy=None, sr=None, sg=None,
        sh=None, sn=None, post=1, pre=1, act=1, rs=1.0, bs=1.0, eps=1e-5, dtype=la.LA_F32, rdtype=la.LA_F32):
    return la.la_block_norm_fwd(y, r, gate, w1, b1, w2, b2, h, n, B, L, d, sy, sr, sg, sh, sn, post, pre, act, rs, bs,
                                eps, dtype, rdtype, None)


def bwd(y=P, r=P, gate=None, w1=None, b1=None, w2=None, b2=None, dh=P, dn=P, dr=P, dy=P, dgate=None, dw1=None, db1=None,
        dw2=None, db2=None, B=2, L=3, d=8, sy=None, sr=None, sg=None, sdh=None, sdn=None, sdr=None, sdy=None, sdg=None,
        post=1, pre=1, act=1, rs=1.0, bs=1.0, eps=1e-5, dtype=la.LA_F32, rdtype=la.LA_F32, ws=None, wsb=0):
    return la.la_block_norm_bwd(y, r, gate, w1, b1, w2, b2, dh, dn, dr, dy, dgate, dw1, db1, dw2, db2, B, L, d, sy, sr,
                                sg, sdh, sdn, sdr, sdy, sdg, post, pre, act, rs, bs, eps, dtype, rdtype, ws, wsb, None)


@pytest.mark.parametrize("call,name", [(fwd, k) for k in ("y", "r", "h")] + [(bwd, k) for k in ("y", "r", "dr", "dy")],
                         ids=lambda v: getattr(v, "__name__", v))
def test_null_pointers(call, name):
    assert call(**{name: None}) == la.LA_ERR_NULL


def test_pointers_that_go_together():
    assert bwd(gate=P) == la.LA_ERR_NULL
    assert bwd(dgate=P) == la.LA_ERR_NULL
    assert bwd(dh=None, dn=None) == la.LA_ERR_NULL
    assert bwd(dn=None, dw2=P) == la.LA_ERR_NULL
    assert bwd(dn=None, db2=P) == la.LA_ERR_NULL


@pytest.mark.parametrize("call", [fwd, bwd])
def test_what_is_refused(call):
    for size in (dict(B=0), dict(L=-1), dict(d=0), dict(B=1 << 30, L=1 << 30, d=1 << 19)):
        assert call(**size) == la.LA_ERR_SHAPE
    for kind in (dict(post=3), dict(post=-1), dict(pre=0), dict(pre=3), dict(act=3), dict(dtype=2), dict(d=8193),
                 dict(dtype=la.LA_F32, rdtype=la.LA_BF16), dict(rdtype=7)):
        assert call(**kind) == la.LA_ERR_UNSUPPORTED
    for arg in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rs=float("inf")),
                dict(bs=float("nan")), dict(sy=st(-8, 8)), dict(sr=st(24, -8)), dict(y=ODD), dict(r=ODD), dict(w1=ODD),
                dict(b2=ODD)):
        assert call(**arg) == la.LA_ERR_ARG


def test_outputs_must_not_fold():
    for s in ("sh", "sn"):
        assert fwd(**{s: st(24, 4)}) == la.LA_ERR_ARG
    for s in ("sdr", "sdy"):
        assert bwd(**{s: st(0, 8)}) == la.LA_ERR_ARG
    assert bwd(gate=P, dgate=P, sdg=st(24, 0)) == la.LA_ERR_ARG


def test_workspace():
    assert la.la_block_norm_bwd_workspace_bytes(2, 3, 8193) == 0
    assert la.la_block_norm_bwd_workspace_bytes(2, 0, 8) == 0
    assert la.la_block_norm_bwd_workspace_bytes(2, 3, 8) > 0


def test_wrappers_refuse():
    x = torch.zeros(1, 3, 8)
    with pytest.raises(ValueError, match="CUDA tensors are needed"):
        la.block_norm_fwd(x, x)
    with pytest.raises(ValueError, match="dgate is given without gate"):
        la.block_norm_bwd(x, x, x, x, dgate=x)
    with pytest.raises(ValueError, match="without a norm"):
        la.block_norm_bwd(x, x, x, x, pre_norm="none")
    with pytest.raises(KeyError):
        la.block_norm_fwd(x, x, post_norm="group")
