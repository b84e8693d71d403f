"""The block norm's gate far out, where its activation or its slope is small: relative to itself.

u = 2^-24.  fp32 gates: with e = exp(-|z|), off by 2 u (the library function's bound is 2 units in the last
place, at most 4 u), the sum 1 + e by 1 u and the quotient by 1 u, the smaller of sigmoid and 1 - sigmoid is e / (1 + e)
to 8 u and the larger 1 / (1 + e) to 4 u.  The slope of the sigmoid is their product: 13 u; that of SiLU, s (1 + z (1 -
s)), is off by (8 + 1) u |z| (1 - s) and 2 u of the sum, relative to its two terms: away from its root 16 u of the
terms.  bf16 gates: e by 2^x in hardware, off by 2^-22 and by its argument's rounding, |z| 2^-23 at most, so
(5 + |z|) 2^-23 of the smaller, next to the output's own 2^-8."""
import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
from gated_reference import HALF, U  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
D = 64


def both(act, dtype, z):
    """h (the activation itself: y 1, residual 0, no norm) and the gate's gradient (the slope) for gates z."""
    z = z.to(dtype).view(1, -1, D)
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    kw = dict(gate=z.cuda(), activation=act, post_norm="none", pre_norm="none")
    h, _ = la.block_norm_fwd(one.cuda(), zero.cuda(), **kw)
    got = la.block_norm_bwd(one.cuda(), zero.cuda(), one.cuda(), None, **kw)
    # the formulas in 64 bits, each in a form that does not cancel
    x = z.double()
    e = torch.exp(-x.abs())
    small, large = e / (1 + e), 1 / (1 + e)
    s, rest = torch.where(x < 0, small, large), torch.where(x < 0, large, small)
    if act == "sigmoid":
        return x, h, got["dgate"], s, s * rest, s * rest, s * rest
    return x, h, got["dgate"], x * s, s * (1 + x * rest), s, s * (x * rest).abs()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_activation_and_slope_relative_to_themselves(act, dtype):
    gen = torch.Generator().manual_seed(1)
    n = 64 * D
    z = torch.exp(torch.rand(n, generator=gen) * 9.0 - 4.6) * torch.where(torch.rand(n, generator=gen) < 0.5, -1.0, 1.0)
    # as far as e^-|z| is in fp32's normal range
    x, h, slope, want, wslope, part, product = both(act, dtype, z.clamp(-86.0, 86.0))
    r = 16 * U if dtype == F32 else (8 + x.abs()) * 2.0 ** -22
    half = HALF[dtype]
    err = (h.double().cpu() - want).abs()
    assert (err <= (r + half) * want.abs()).all(), float((err / want.abs()).max())
    err = (slope.double().cpu() - wslope).abs()
    terms = part + product if act == "silu" else wslope
    assert (err <= r * terms + half * wslope.abs() + U * terms).all(), float((err / terms).max())


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_below_the_normal_range(act):
    """e^-|z| below the normal range of fp32, down to its last steps: off by such a step (2^-149) as well."""
    z = -torch.linspace(87.0, 103.0, 4 * D)
    x, h, slope, want, wslope, _, _ = both(act, F32, z)
    step = 2.0 ** -149 * 2
    for got, w in ((h, want), (slope, wslope)):
        err = (got.double().cpu() - w).abs()
        far = x.abs() if act == "silu" else 1.0
        assert (err <= 32 * U * w.abs() + step * (far + 1)).all(), float((err / w.abs()).max())
