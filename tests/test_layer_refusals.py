"""Refusals of the torch wrappers around the attention that need no GPU."""
import pytest

import chunkwise_causal_linear_gb300 as la
from chunkwise_causal_linear_gb300 import build as la_build


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    la_build.build()
    return torch


def test_outputs_without_their_inputs(torch):
    """An output tensor that the call would not write is refused, as the C ABI refuses it."""
    x = torch.zeros(1, 1, 1, 8)
    table = la.RotaryTable(torch.zeros(4, dtype=torch.int64), 8)
    with pytest.raises(ValueError, match="k_out is given without k"):
        la.rotary(x, None, table, k_out=torch.zeros_like(x))
    with pytest.raises(ValueError, match="dgate is given without gate"):
        la.group_norm_bwd(x, x[:, 0], dgate=torch.zeros(1, 1, 8))
