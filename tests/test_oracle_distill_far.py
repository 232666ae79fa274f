"""The 64-bit distillation loss of rows far from zero."""
import numpy as np
import pytest

from oracle import logits as L


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("size", [0.0, 1e12, 1e20, -1e20, -3.3895313892515355e38])
def test_rows_far_from_zero(tail, size):
    """Equal logits give the loss of the uniform row, wherever they lie."""
    rng = np.random.default_rng(9)
    z = rng.normal(0, 2, 40)
    ids = np.array([3, 4, 17])
    lse = L.logsumexp(z) if tail else None
    want = L.distill_row(np.zeros(40), ids, z[ids], 1.0, lse)
    got = L.distill_row(np.full(40, size), ids, z[ids], 1.0, lse)
    assert abs(got[0] - want[0]) < 1e-14 and np.abs(got[1] - want[1]).max() < 1e-15
