"""Sums of log decays past every number that a product of decays could still be told from 0 by: segments of few
heads on the tensor cores whose rows decay fast, one of them growing (none is left out of the sums then)."""
import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
from gated_reference import U  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def few_heads(rows):
    """H heads and L rows for segments of `rows` rows: a third of the SMs' number of heads is cut in three."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return sms // 3, 3 * rows


@pytest.mark.parametrize("rows,rate", [(4096, -103.0), (8192, -50.0), (8192, -60.0), (4096, -3.0)])
def test_fast_decays_and_a_growing_row(rows, rate):
    """2^19 doublings are 363,409 nats: 4096 rows of -103 and 8192 of -50 or -60 are more, of -3 fewer.  A row's
    decay leaves e^-50 at most (e^-3 in the last case) of what is before: the formula is that of the fp32 path,
    and rows are off by what operands rounded to bf16 allow."""
    H, L = few_heads(rows)
    d = 64
    gen = torch.Generator("cuda").manual_seed(rows)
    q, k, v, do = (torch.randn(1, H, L, d, generator=gen, device="cuda").to(BF16) for _ in range(4))
    s0, ds = (torch.randn(1, H, d, d, generator=gen, device="cuda") for _ in range(2))
    g = torch.full((1, H, L), rate, device="cuda")
    g[:, :, 100::rows] = 0.01
    kw = dict(scale=0.2, state0=s0)
    out, state = la.gated_fwd(q, k, v, g, path=la.LA_PATH_TC, **kw)
    want, wstate = la.gated_fwd(q, k, v, g, path=la.LA_PATH_SIMT, **kw)
    assert la.la_last_device_status(None) == la.LA_OK
    # terms' magnitudes: the row's own pair, and the one before the growing row; the others are below e^-3 of them
    a = q.float().abs().mul(k.float().abs()).sum(-1, keepdim=True) * v.float().abs() * 0.2
    size = a + a.mean()
    assert torch.isfinite(out).all() and torch.isfinite(state).all()
    # two operands rounded by 2^-8, and both outputs
    assert ((out.float() - want.float()).abs() <= 3 * 2.0 ** -8 * size + 2.0 ** -7 * want.float().abs() + 1e-3 * size.mean()).all()
    assert ((state - wstate).abs() <= 6 * d * U * (wstate.abs() + wstate.abs().mean())).all()
    got = la.gated_bwd(q, k, v, g, do, dstate=ds, path=la.LA_PATH_TC, **kw)
    ref = la.gated_bwd(q, k, v, g, do, dstate=ds, path=la.LA_PATH_SIMT, **kw)
    assert la.la_last_device_status(None) == la.LA_OK
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dstate0"), got, ref):
        assert torch.isfinite(x).all(), name
        err = float((x.double() - y.double()).square().mean().sqrt())
        # three roundings of half a step of bf16, two outputs'; dg and dstate0 fp32 sums of about 6 d roundings
        most = (2 * 2.0 ** -8 if x.dtype == BF16 else (6 * 3 * d) ** 0.5 * 2 * U * d) * float(y.double().square().mean().sqrt())
        # e^-103 is below fp32's normal range (2^-126 = e^-87.3), where a value is held to a step of 2^-149 or flushed to 0:
        # what such a decay alone leaves (dstate0 and most of dg) may be off by all of itself, 2^-126 at most
        assert err <= most + 2.0 ** -126, (name, err, most)
