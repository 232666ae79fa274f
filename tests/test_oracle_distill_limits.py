"""The distillation loss where its last term is left out: the 64-bit
implementation's gradient against differences of its loss."""
import numpy as np
import pytest

from oracle import logits as L


def slopes(x, ids, z, temp, lse, h=1e-5):
    g = np.zeros(len(x))
    for v in np.flatnonzero(x > -np.inf):
        d = np.zeros(len(x))
        d[v] = h
        g[v] = (L.distill_row(x + d, ids, z, temp, lse)[0] - L.distill_row(x - d, ids, z, temp, lse)[0]) / (2 * h)
    return g


@pytest.mark.parametrize("temp", [0.7, 2.0])
@pytest.mark.parametrize("how", ["no logit off the list", "probabilities above one", "everything listed"])
def test_gradient_without_the_last_term(how, temp):
    """sum p = b is not one there, and the softmax in the gradient is scaled by it."""
    rng = np.random.default_rng(8)
    x, z = rng.normal(0, 2, 12), rng.normal(0, 2, 12)
    ids = np.arange(12) if how == "everything listed" else np.array([1, 4, 6, 9])
    true = L.logsumexp(z[ids] / temp)
    lse = true - 0.3 if how == "probabilities above one" else true + 0.8
    if how == "no logit off the list":
        off = np.ones(12, bool)
        off[ids] = False
        x[off] = -np.inf
    loss, grad, q, p, P, Q = L.distill_row(x, ids, z[ids], temp, lse)
    assert abs(p.sum() - 1) > 0.2
    # central differences: off by h^2 times a third derivative below 2 sum p / T^3, and by 1e-15 / h
    assert np.abs(slopes(x, ids, z[ids], temp, lse) - grad).max() < 4e-10 / temp ** 3 + 1e-9
    assert abs(grad.sum()) < 1e-14  # the softmax of shifted rows is the same
