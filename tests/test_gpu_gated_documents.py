"""The decays' gradient of packed documents: what lies behind a -inf is not part of the sums before it, neither its
roundings nor its infinities and NaN."""
import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
import gated_reference as ref  # noqa: E402
from gated_reference import close  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def grads(x, **kw):
    q, k, v, g, s0, n, do, ds = (t if t is None else t.cuda() for t in x)
    return la.gated_bwd(q, k, v, g, do, scale=0.2, state0=s0, lengths=n, dstate=ds, **kw)


# one sum of 1024 rows and several; resets next to one another, on both sides of the sums' steps of 1024 and 4 rows
CUTS = [(150, (60,)), (150, (1, 2, 3, 4, 77, 149)), (1100, (23, 24, 512, 1024)), (1100, (75, 76, 77, 78, 79, 1023)), (2300, (0, 252, 1276, 2299))]


@TYPES
@pytest.mark.parametrize("L,cuts", CUTS, ids=lambda v: str(v).replace(" ", ""))
def test_documents_of_different_size(L, cuts, dtype):
    """Each document's gradients of its decays are off by roundings of its own terms, when the next one's are 2^16
    times as large.  The bound is that of a sequence alone (test_gpu_gated.py), without the rows of others."""
    d = 64
    q, k, v, g, s0, _, do, ds = ref.draw(1, 2, 2, L, d, d, dtype, "token", True, seed=L + len(cuts), resets=0)
    g[:, :, list(cuts)] = float("-inf")
    edges = sorted({0, *cuts, L})
    # the bf16 path's products keep 24 bits of each document's rows: documents begin on chunks of their own only by
    # chance, so the factors are powers of two, which change no rounding
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        do[:, :, a:b] *= 2.0 ** (16 * (i % 2))
    ds = ds * 2.0 ** (16 * ((len(edges) - 2) % 2))
    x = (q, k, v, g, s0, None, do, ds)
    got = grads(x)[3].cpu()
    m = ref.magnitudes(q, k, v, g, 0.2, s0, None, do, ds)
    want = ref.backward(q, k, v, g, do, 0.2, s0, None, ds)["dg"]
    steps = 6 * (L + 2 * d)
    for a, b in zip(edges, edges[1:]):
        size = m["dg"][:, :, a:b]
        size = size + size.mean(-1, keepdim=True)
        if b == L:
            size = size + m["end"][..., None]
        close(f"dg {a}:{b}", got[:, :, a:b], want[:, :, a:b], size, F32, steps)
    for c in cuts:
        assert not got[:, :, c].any()


@TYPES
@pytest.mark.parametrize("L", [200, 700, 1500])
def test_a_bad_row_of_a_later_document(L, dtype):
    """Bit for bit, where the bad row's chunk of 64 is another than the reset's (any row in fp32)."""
    d = 64
    q, k, v, g, s0, _, do, ds = ref.draw(1, 2, 1, L, d, d, dtype, "token", True, seed=L, resets=0)
    for cut, bad in ((64, 128), (20, 64), (100, 190), (63, L - 1)):
        g2 = g.clone()
        g2[:, :, cut] = float("-inf")
        want = grads((q, k, v, g2, s0, None, do, ds))[3]
        for value in (float("nan"), float("inf")):
            spoilt = [t.clone() for t in (q, k, v, do)]
            for t in spoilt:
                t[:, :, bad, ::5] = value
            got = grads((*spoilt[:3], g2, s0, None, spoilt[3], ds))[3]
            assert torch.equal(got[:, :, :cut + 1], want[:, :, :cut + 1]), (cut, bad, value)
        got = grads((q, k, v, g2, s0, None, do, torch.full_like(ds, float("nan"))))[3]
        if cut // 64 < L // 64:
            assert torch.equal(got[:, :, :cut + 1], want[:, :, :cut + 1]), cut


@TYPES
@pytest.mark.parametrize("L", [200, 700, 1500])
def test_a_bad_row_or_state_before(L, dtype):
    """The rows from a reset on, when a row of an earlier document or the first state is bad."""
    d = 64
    q, k, v, g, s0, _, do, ds = ref.draw(1, 2, 1, L, d, d, dtype, "token", True, seed=L + 1, resets=0)
    for bad, cut in ((None, 0), (None, 1), (None, 37), (5, 64), (63, 84), (5, 130), (100, L - 3)):
        g2 = g.clone()
        g2[:, :, cut] = float("-inf")
        want = grads((q, k, v, g2, s0, None, do, ds))[3]
        for value in (float("nan"), float("inf")):
            spoilt = [t.clone() for t in (q, k, v, do)]
            for t in spoilt:
                if bad is not None:
                    t[:, :, bad, ::5] = value
            first = s0 if bad is not None else torch.full_like(s0, value)
            got = grads((*spoilt[:3], g2, first, None, spoilt[3], ds))[3]
            assert torch.equal(got[:, :, cut:], want[:, :, cut:]), (bad, cut, value)


@TYPES
def test_rows_behind_the_end_and_resets(dtype):
    """Padded sequences with resets, the gradient of a decay per token: as the 64-bit recurrence's, and 0 at resets."""
    B, H, L, d = 4, 2, 300, 64
    q, k, v, g, s0, n, do, ds = ref.draw(B, H, H, L, d, d, dtype, "token", True, True, seed=5, resets=0.1)
    x = (q, k, v, g, s0, n, do, ds)
    got = grads(x)[3].cpu()
    m = ref.magnitudes(q, k, v, g, 0.2, s0, n, do, ds)
    want = ref.backward(q, k, v, g, do, 0.2, s0, n, ds)["dg"]
    size = m["dg"] + m["dg"].mean(-1, keepdim=True) + m["end"][..., None]
    close("dg", got, want, size, F32, 6 * (L + 2 * d))
    assert not got[torch.isneginf(g)].any()
