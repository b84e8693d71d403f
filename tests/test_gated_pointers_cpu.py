"""Pointers of the gated attention's integers that are not on 4 bytes are refused on the host."""
import pytest

pytest.importorskip("torch")

import chunkwise_causal_linear_gb300 as la  # noqa: E402
from test_gated_cpu import ODD, P, _lib, bwd, fwd, step  # noqa: E402, F401


def test_lengths_and_slots():
    assert fwd(lengths=ODD) == la.LA_ERR_ARG
    assert bwd(lengths=ODD) == la.LA_ERR_ARG
    assert fwd(slots=ODD, s0=P, n=4) == la.LA_ERR_ARG
    assert step(slots=ODD, n=4) == la.LA_ERR_ARG
