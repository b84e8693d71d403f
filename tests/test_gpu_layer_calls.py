"""Calls of the operators around the attention at the same time: host threads with streams and buffers
of their own."""
import threading

import numpy as np
import pytest

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


def at_once(calls, n):
    """Each of the calls n times in a thread of its own; the statuses that are not 0."""
    bad = []
    start = threading.Barrier(len(calls))

    def run(call):
        start.wait()
        for _ in range(n):
            rc = call()
            if rc:
                bad.append(rc)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return bad


def test_group_norm_of_different_widths_at_once(la):
    """One kernel, whose shared memory depends on the width, launched by threads with different ones."""
    import torch
    rng = np.random.default_rng(50)
    held, calls, wants = [], [], []
    for d in (6017, 6019, 8191, 8189):
        x, dout = (torch.from_numpy(rng.normal(size=(1, 1, 2, d))).to(torch.bfloat16).cuda() for _ in range(2))
        w = torch.from_numpy(rng.normal(size=d)).float().cuda()
        wants.append(la.group_norm_bwd(x, dout.view(1, 2, d), w))
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws = torch.empty(la.la_group_norm_bwd_workspace_bytes(1, 1, 2, d), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        held.append((x, dout, w, dx, dw, ws, stream))

        def call(d=d, x=x, dout=dout, w=w, dx=dx, dw=dw, ws=ws, stream=stream):
            return la.la_group_norm_bwd(x.data_ptr(), w.data_ptr(), None, None, dout.data_ptr(), dx.data_ptr(), None,
                                        dw.data_ptr(), None, 1, 1, 2, d, None, None, None, None, None, 1, la.LA_ACT_SILU,
                                        1e-5, la.LA_BF16, ws.data_ptr(), ws.numel(), stream.cuda_stream)

        calls.append(call)
    torch.cuda.synchronize()
    assert at_once(calls, 3000) == []
    torch.cuda.synchronize()
    for (_, _, _, dx, dw, _, _), want in zip(held, wants):
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[2])


def test_recurrences_at_once(la):
    """Threads that launch the same kernel in clusters, each on a stream of its own."""
    import torch
    x = torch.randn(1, 2, 3000, 64, device="cuda")
    outs, calls = [], []
    for _ in range(4):
        out, stream = torch.empty_like(x), torch.cuda.Stream()
        outs.append((out, stream))

        def call(out=out, stream=stream):
            return la.la_recurrence_fwd(x.data_ptr(), x.data_ptr(), None, None, out.data_ptr(), None, None, *x.shape,
                                        None, None, None, la.LA_GATE_SIGMOID, 1, la.LA_F32, la.LA_F32,
                                        stream.cuda_stream)

        calls.append(call)
    torch.cuda.synchronize()
    assert at_once(calls, 200) == []
    torch.cuda.synchronize()
    want = la.recurrence_fwd(x, x, complement=True)[0]
    assert all(torch.equal(out, want) for out, _ in outs)
