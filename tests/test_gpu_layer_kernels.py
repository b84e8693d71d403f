"""Every kernel that the dispatch of the operators around the attention can choose: vector widths,
threads of a group, alignments, broadcast inputs, strided views on all sides."""
import numpy as np
import pytest

import layer_reference as ref
from test_gpu_layer import check, dev, gate_values, host, run_recurrence, strided

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


def shifted(t):
    """A contiguous copy that starts one element into its storage."""
    import torch
    v = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    v.copy_(t)
    return v


# ---- recurrence: the forward kernel with two channels a lane (bf16, enough heads, even d > 32) ------
@pytest.mark.parametrize("kind", ["value", "log", "sigmoid"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("d", [34, 64, 66, 100, 128])
def test_two_channels_a_lane(la, kind, complement, d):
    run_recurrence(la, (2, 80, 150, d), kind, complement, "bf16", "bf16", seed=30)


@pytest.mark.parametrize("order", [None, "blh"])
@pytest.mark.parametrize("d", [36, 64, 130])
@pytest.mark.parametrize("lengths", [[0, 1, 300], [128, 129, 127], [-5, 1000, 256]])
def test_two_channels_a_lane_padded_and_strided(la, order, d, lengths):
    run_recurrence(la, (3, 52, 300, d), "sigmoid", True, "bf16", "bf16", order=order, lengths=lengths, seed=31)
    run_recurrence(la, (3, 52, 300, d), "value", False, "bf16", "bf16", order=order, lengths=lengths, initial=False,
                   seed=32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2, 700, 64), (2, 80, 150, 64), (1, 3, 300, 33)], ids=str)
def test_recurrence_off_a_vector_boundary(la, dtype, shape):
    """Every tensor one element into its storage: the copies are 4 or 2 bytes."""
    rng = np.random.default_rng(33)
    B, H, L, d = shape
    x, do = dev(rng.normal(size=shape), dtype), dev(rng.normal(size=shape), dtype)
    g = dev(gate_values(rng, "log", shape), dtype)
    kw = dict(gate_kind="log", complement=True)
    out, last, chunks = la.recurrence_fwd(shifted(x), shifted(g), out=shifted(x), save_chunks=True, **kw)
    dx, dg, dh0 = la.recurrence_bwd(shifted(x), shifted(g), chunks, shifted(do), dx=shifted(x), dgate=shifted(g), **kw)
    hx, hg, hd = host(x), host(g), host(do)
    want, wlast, _ = ref.recurrence(hx, hg, "log", True)
    bound = ref.recurrence_bounds(hx, hg, "log", True)
    check("out", out, want, bound, dtype)
    check("last", last, wlast, bound[:, :, -1])
    wx, wg, w0, _ = ref.recurrence_grads(hx, hg, hd, None, "log", True)
    bx, bg, b0 = ref.recurrence_grad_bounds(hx, hg, hd, None, "log", True)
    check("dx", dx, wx, bx, dtype)
    check("dg", dg, wg, bg, dtype)
    check("dh0", dh0, w0, b0)


# ---- broadcast inputs: equal to their copies, bit for bit ---------------------------------------------
def spread(shape, axes, rng, dtype):
    """A tensor of that shape with stride 0 along the axes."""
    import torch
    t = dev(rng.normal(size=[1 if i in axes else n for i, n in enumerate(shape)]), dtype).expand(shape)
    assert all(t.stride(i) == 0 for i in axes)
    return t


@pytest.mark.parametrize("axes", [(0,), (1,), (2,), (0, 1), (0, 1, 2)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 3, 700, 64), (2, 80, 70, 64)], ids=str)
def test_broadcast_inputs(la, axes, dtype, shape):
    import torch
    rng = np.random.default_rng(34)
    B, H, L, d = shape
    x, g, do = (spread(shape, axes, rng, dtype) for _ in range(3))

    def equal(got, want):
        assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)

    full = [t.contiguous() for t in (x, g, do)]
    got, want = (la.recurrence_fwd(t[0], t[1], save_chunks=True) for t in ((x, g), full))
    equal(got, want)
    equal(la.recurrence_bwd(x, g, got[2], do), la.recurrence_bwd(full[0], full[1], got[2], full[2]))
    table = la.rotary_table(d)
    equal(la.rotary(x, g, table), la.rotary(full[0], full[1], table))
    rows = tuple({0: 0, 2: 1}[a] for a in axes if a != 1)
    gate, dout = (spread((B, L, H * d), rows, rng, dtype) for _ in range(2))
    w = dev(rng.normal(size=H * d))
    equal([la.group_norm_fwd(x, w, gate=gate)], [la.group_norm_fwd(full[0], w, gate=gate.contiguous())])
    equal(la.group_norm_bwd(x, dout, w, gate=gate),
          la.group_norm_bwd(full[0], dout.contiguous(), w, gate=gate.contiguous()))


# ---- rotary: vectors of 8, 4 and 1 elements of bf16, 4 and 1 of fp32 -----------------------------------
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,rot", [(8, 8), (24, 24), (64, 40), (72, 8), (20, 16), (78, 38), (68, 24), (100, 96)])
@pytest.mark.parametrize("move", [False, True])
def test_rotary_vectors(la, layout, dtype, d, rot, move):
    import torch
    rng = np.random.default_rng(35)
    B, H, Hk, L = 2, 3, 2, 9
    q, k = dev(rng.normal(size=(B, H, L, d)), dtype), dev(rng.normal(size=(B, Hk, L, d)), dtype)
    pos = rng.integers(0, 5000, size=(B, L)).astype(np.int32)
    table, theta = la.rotary_table(rot), ref.frequencies(rot)
    kw = dict(positions=torch.from_numpy(pos).cuda(), layout=layout)
    a, b = (shifted(q), shifted(k)) if move else (strided(q, "blh"), strided(k, "blh"))
    for inverse in (False, True):
        for outs in ({}, dict(q_out=shifted(q), k_out=shifted(k))):
            qo, ko = la.rotary(a, b, table, inverse=inverse, **kw, **outs)
            for got, src in ((qo, q), (ko, k)):
                want, bound = ref.rotary(host(src), pos, theta, layout, inverse)
                check("rotary", got, want, bound, dtype)
                assert torch.equal(got[..., rot:], src[..., rot:])


# ---- group norm: single elements, pairs and 16-byte vectors by the threads of a group -----------------
ODD = [2, 3, 31, 33, 65, 129, 257, 1023, 1025, 8191]  # single elements
EVEN = [10, 66, 130, 258, 514, 2050, 8190]  # pairs in bf16, single elements in fp32
WHOLE = [8, 16, 24, 28, 264, 512, 520, 768, 1032, 2056, 4104, 8192]  # vectors (28: of fp32 alone)


def padded(t):
    """The same values as a view of rows eight elements longer, the rest NaN."""
    import torch
    rows = torch.full((*t.shape[:-1], t.shape[-1] + 8), float("nan"), dtype=t.dtype, device=t.device)
    rows[..., :t.shape[-1]] = t
    return rows[..., :t.shape[-1]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("d", ODD + EVEN + WHOLE)
def test_group_norm_sizes(la, dtype, gated, d):
    import torch
    rng = np.random.default_rng(36)
    B, H, L = (2, 2, 37) if d <= 600 else (1, 2, 3)
    x = dev(rng.normal(size=(B, H, L, d)) + 0.3, dtype)
    w, b = dev(rng.normal(size=H * d)), dev(rng.normal(size=H * d))
    gate = dev(rng.normal(size=(B, L, H * d)) * 2, dtype) if gated else None
    dout = dev(rng.normal(size=(B, L, H * d)), dtype)
    r = ref.group_norm(host(x), host(w).reshape(H, d), host(b).reshape(H, d),
                       host(gate).reshape(B, L, H, d) if gated else None, 1e-5, "silu", True,
                       host(dout).reshape(B, L, H, d))
    # as they are, as views of longer rows, and one element off
    for view in (lambda t: t, padded, shifted):
        z, blank = view(gate) if gated else None, torch.zeros_like(dout)
        out = la.group_norm_fwd(view(x), w, b, gate=z, out=view(blank))
        check("out", out, *r["out"], dtype)
        dx, dgate, dw, db = la.group_norm_bwd(view(x), view(dout), w, b, gate=z, dx=view(torch.zeros_like(x)),
                                              dgate=view(blank) if gated else None)
        check("dx", dx.transpose(1, 2), *r["dx"], dtype)
        if gated:
            check("dgate", dgate, *r["dgate"], dtype)
        check("dw", dw, *r["dw"])
        check("db", db, *r["db"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_group_norm_leaves_the_rest_of_a_row(la, dtype):
    """What stands between the rows of a strided output stays."""
    import torch
    rng = np.random.default_rng(37)
    B, H, L, d = 2, 3, 41, 64
    x, gate = dev(rng.normal(size=(B, H, L, d)), dtype), dev(rng.normal(size=(B, L, H * d)), dtype)
    rows = torch.full((B, L, H * d + 8), 7.0, dtype=x.dtype, device="cuda")
    la.group_norm_fwd(x, gate=gate, out=rows[..., :H * d])
    assert (rows[..., H * d:] == 7).all() and torch.equal(rows[..., :H * d], la.group_norm_fwd(x, gate=gate))
