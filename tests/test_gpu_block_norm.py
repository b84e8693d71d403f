"""The norms around a block on the GPU against their definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
from gated_reference import HALF, U  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def norm(x, kind, w, b):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    if kind != "none":
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * w if w is not None else x
    return x + b if b is not None else x


def act_of(z, kind):
    return z if kind == "none" else torch.sigmoid(z) * (z if kind == "silu" else 1.0)


def reference(p, post, pre, act, rs, bs, dh=None, dn=None):
    """h, n and, with dh and dn, the gradients, of 64-bit copies of the tensors of p."""
    x = {k: v.detach().double().cpu().requires_grad_() for k, v in p.items() if v is not None}
    u = norm(x["y"], post, x.get("post_w"), x.get("post_b"))
    h = rs * x["r"] + bs * u * (act_of(x["gate"], act) if "gate" in x else 1.0)
    n = norm(h, pre, x.get("pre_w"), x.get("pre_b")) if pre != "none" else None
    outs = {"h": h.detach(), "n": None if n is None else n.detach()}
    if dh is None and dn is None:
        return outs
    loss = 0
    if dh is not None:
        loss = loss + (h * dh.double().cpu()).sum()
    if dn is not None:
        loss = loss + (n * dn.double().cpu()).sum()
    grads = torch.autograd.grad(loss, list(x.values()), allow_unused=True)
    return outs | {"d" + k: g for k, g in zip(x, grads)}


def draw(B, L, d, dtype, rdtype, gated, post, pre, affine=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    p = dict(y=n(B, L, d).to(dtype), r=(2 * n(B, L, d)).to(rdtype), gate=n(B, L, d).to(dtype) if gated else None,
             post_w=1 + 0.2 * n(d) if affine else None, post_b=0.2 * n(d) if affine and post == "layer" else None,
             pre_w=1 + 0.2 * n(d) if affine and pre != "none" else None, pre_b=0.2 * n(d) if affine and pre == "layer" else None)
    p = {k: v if v is None else v.cuda() for k, v in p.items()}
    dh, dn = n(B, L, d).to(rdtype).cuda(), n(B, L, d).to(dtype).cuda()
    return p, dh, dn if pre != "none" else None


def args(p, post, pre, act, rs, bs):
    return dict(gate=p["gate"], activation=act, post_norm=post, post_weight=p["post_w"], post_bias=p["post_b"],
                pre_norm=pre, pre_weight=p["pre_w"], pre_bias=p["pre_b"], residual_scale=rs, branch_scale=bs, eps=EPS)


def row_close(name, got, want, d):
    """Each value meets fewer than 40 roundings of its own, and those of the row's sums, d of them in groups:
    64 U of the row's largest magnitude in all, next to half a step of its type (a bf16 sigmoid is taken to
    2^-21)."""
    err = (got.double().cpu() - want).abs()
    scale = want.abs().amax(-1, keepdim=True) + 1.0
    extra = 64 * U * scale if got.dtype == F32 else 2.0 ** -18 * scale
    bad = err > HALF[got.dtype] * want.abs() + extra
    assert not bad.any(), (name, float((err / scale).max()))


def sum_close(name, got, want, terms):
    """Sums over the rows: `terms` is the sum of the terms' magnitudes, each off by 64 U or, with bf16's
    sigmoid, 2^-18, and roundings of the sums, one per row of a group and per group."""
    err = (got.double().cpu() - want).abs()
    assert not (err > 2.0 ** -17 * terms).any(), (name, float((err / terms).max()))
    rms = lambda x: float(x.square().mean().sqrt())  # noqa: E731
    assert rms(err) <= 2e-6 * rms(terms)


def check(B, L, d, dtype, rdtype, gated, post, pre, act="silu", affine=True, rs=1.0, bs=0.5, seed=0):
    p, dh, dn = draw(B, L, d, dtype, rdtype, gated, post, pre, affine, seed)
    kw = args(p, post, pre, act, rs, bs)
    h, n = la.block_norm_fwd(p["y"], p["r"], **kw)
    got = la.block_norm_bwd(p["y"], p["r"], dh, dn, **kw)
    want = reference(p, post, pre, act, rs, bs, dh, dn)
    row_close("h", h, want["h"], d)
    if pre == "none":
        assert n is None
    else:
        row_close("n", n, want["n"], d)
    for name in ("dy", "dr", "dgate"):
        if got[name] is not None:
            row_close(name, got[name], want[name], d)
        else:
            assert name == "dgate" and not gated
    rows = B * L
    for name in ("post_w", "post_b", "pre_w", "pre_b"):
        if p[name] is None:
            assert got["d" + name] is None
        else:
            # terms of the sums: unit-sized gradients times normalised values
            terms = rows ** 0.5 * want["d" + name].abs().clamp_min(1.0) + rows * 1.0
            sum_close("d" + name, got["d" + name], want["d" + name], terms)


TYPES = [(F32, F32), (BF16, F32), (BF16, BF16)]


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("d", [1, 7, 8, 40, 255, 256, 264, 512, 768, 1000, 1024, 2048, 2056, 3000, 4096, 8184, 8191, 8192])
def test_widths(d, types):
    check(2, 5, d, *types, True, "rms", "layer", seed=d)
    check(3, 3, d, *types, False, "layer", "rms", seed=d + 1)


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_kinds(post, pre, types):
    for act in ("none", "silu", "sigmoid"):
        check(2, 9, 136, *types, True, post, pre, act, seed=3)
    check(1, 9, 300, *types, False, post, pre, affine=False, rs=0.7, bs=-1.5, seed=4)


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 2048), (700, 1, 96), (3, 1111, 400), (2, 3000, 33)], ids=lambda s: "x".join(map(str, s)))
def test_many_rows(size, types):
    check(*size, *types, True, "rms", "rms", seed=5)


def test_only_one_gradient():
    """dn or dh alone."""
    p, dh, dn = draw(2, 6, 64, F32, F32, True, "rms", "rms")
    kw = args(p, "rms", "rms", "silu", 1.0, 1.0)
    for a, b in ((dh, None), (None, dn)):
        got = la.block_norm_bwd(p["y"], p["r"], a, b, **kw)
        want = reference(p, "rms", "rms", "silu", 1.0, 1.0, a, b)
        for name in ("dy", "dr", "dgate"):
            row_close(name, got[name], want[name], 64)
        assert (got["dpre_w"] is None) == (b is None)


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 1300, 500), (2, 1300, 520), (3, 1100, 768), (1, 1300, 1001), (1, 1000, 1504), (1, 700, 2003), (1, 400, 4001),
                                  (1, 333, 5001)], ids=lambda s: "x".join(map(str, s)))
def test_several_rows_a_group(size, types):
    """Every split of a row over threads, each group with more than one row."""
    check(*size, *types, True, "rms", "layer", seed=6)


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16-f32", "bf16"])
def test_views_in_place_and_broadcast(types):
    """Views of wider rows, odd offsets, in place, and one gate for all rows (stride 0)."""
    B, L, d = 2, 70, 256
    p, dh, dn = draw(B, L, d, *types, True, "layer", "layer", seed=6)
    kw = args(p, "layer", "layer", "silu", 1.0, 1.0)
    h, n = la.block_norm_fwd(p["y"], p["r"], **kw)
    grads = la.block_norm_bwd(p["y"], p["r"], dh, dn, **kw)
    for pad, off in ((64, 32), (3, 1)):
        wide = {k: torch.full((B, L, d + pad), 9.0, dtype=x.dtype, device="cuda") for k, x in
                dict(y=p["y"], r=p["r"], gate=p["gate"], h=h, n=n, dr=h, dy=n, dgate=n, dh=dh, dn=dn).items()}
        v = {k: x[..., off:off + d] for k, x in wide.items()}
        for k in ("y", "r", "gate"):
            v[k].copy_(p[k])
        v["dh"].copy_(dh)
        v["dn"].copy_(dn)
        kw2 = kw | dict(gate=v["gate"])
        la.block_norm_fwd(v["y"], v["r"], h=v["h"], n=v["n"], **kw2)
        got = la.block_norm_bwd(v["y"], v["r"], v["dh"], v["dn"], dr=v["dr"], dy=v["dy"], dgate=v["dgate"], **kw2)
        if off == 32:  # the same kernel: the same bits
            assert torch.equal(v["h"], h) and torch.equal(v["n"], n)
            assert all(torch.equal(got[k], grads[k]) for k in grads if grads[k] is not None)
        want = reference(p, "layer", "layer", "silu", 1.0, 1.0, dh, dn)
        for name, x in (("h", v["h"]), ("n", v["n"]), ("dy", got["dy"]), ("dr", got["dr"]), ("dgate", got["dgate"])):
            row_close(name, x, want[name], d)
        for k in ("h", "n", "dr", "dy", "dgate"):  # nothing outside the views
            assert (wide[k][..., :off] == 9).all() and (wide[k][..., off + d:] == 9).all()
    y, r = p["y"].clone(), p["r"].clone()
    la.block_norm_fwd(y, r, h=r, n=y, **kw)
    assert torch.equal(r, h) and torch.equal(y, n)
    a, b = dh.clone(), dn.clone()
    got = la.block_norm_bwd(p["y"], p["r"], a, b, dr=a, dy=b, **kw)
    assert torch.equal(a, grads["dr"]) and torch.equal(b, grads["dy"]) and torch.equal(got["dgate"], grads["dgate"])
    one = p["gate"][:1, :1].expand(B, L, d)
    full = one.contiguous()
    x, z = (la.block_norm_fwd(p["y"], p["r"], **(kw | dict(gate=g))) for g in (one, full))
    assert torch.equal(x[0], z[0]) and torch.equal(x[1], z[1])


def test_rows_of_zeros_and_gates_far_out():
    """A row of zeros is normalised by eps alone; gates far out give 0 or themselves, no NaN."""
    B, L, d = 1, 4, 64
    y = torch.zeros(B, L, d, device="cuda")
    gate = torch.tensor([-1e4, -100.0, 100.0, 1e4], device="cuda")[None, :, None].expand(B, L, d).contiguous()
    for dtype in (F32, BF16):
        p = dict(y=(y + (torch.arange(d, device="cuda") % 3 - 1)).to(dtype), r=y.to(dtype), gate=gate.to(dtype), post_w=None,
                 post_b=None, pre_w=None, pre_b=None)
        h, n = la.block_norm_fwd(p["y"], p["r"], gate=p["gate"], eps=EPS)
        want = reference(p, "rms", "rms", "silu", 1.0, 1.0)
        row_close("h", h, want["h"], d)
        row_close("n", n, want["n"], d)
        h, n = la.block_norm_fwd(y.to(dtype), y.to(dtype))
        assert not h.any() and not n.any()
        got = la.block_norm_bwd(y.to(dtype), y.to(dtype), p["y"], p["y"], gate=p["gate"])
        assert all(torch.isfinite(x).all() for x in got.values() if x is not None)


def test_captured_and_on_another_stream():
    p, dh, dn = draw(3, 50, 768, BF16, F32, True, "rms", "layer", seed=7)
    kw = args(p, "rms", "layer", "silu", 1.0, 1.0)

    def call(stream=None):
        h, n = la.block_norm_fwd(p["y"], p["r"], stream=stream, **kw)
        return [h, n, *[x for x in la.block_norm_bwd(p["y"], p["r"], dh, dn, stream=stream, **kw).values() if x is not None]]

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        call()
    warm.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    p["y"].mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    want = call()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        named = call(side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(named, want))
