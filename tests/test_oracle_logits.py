"""The 64-bit implementations of the logit operators on small cases worked
out by hand, and the gradient against differences of the loss."""
import math

import numpy as np
import pytest

from oracle import logits as L


def test_shape_row_by_hand():
    x = [2.0, -2.0, 4.0, 0.0, 1.0]
    z, _ = L.shape_row(x, prompt=[1, 0], made=[2, 2, 3], rep=2.0, freq=0.5, pres=0.25, temp=0.5,
                       bias=[(4, 3.0), (0, -1.0)], allowed=[True, True, True, True, False])
    # 0: 2/2 - 1; 1: -2*2; 2: 4/2 - 0.5*2 - 0.25; 3: 0 - 0.5 - 0.25; 4: masked
    assert z.tolist() == [0.0, -8.0, 1.5, -1.5, -math.inf]


def test_shape_row_mask_covers_nan_and_inf():
    z, _ = L.shape_row([math.nan, math.inf, -math.inf], allowed=[False, False, False])
    assert (z == -math.inf).all()


def test_top_row_ties_go_to_the_lowest_id():
    st, ids, z, lse = L.top_row([1.0, 3.0, 3.0, -math.inf, 3.0], 2)
    assert st == L.ST_OK and ids.tolist() == [1, 2] and z.tolist() == [3.0, 3.0]
    assert abs(lse - math.log(3 * math.exp(3) + math.exp(1))) < 1e-14
    assert L.top_row([1.0, -math.inf], 2)[1].tolist() == [0]
    assert L.top_row([-math.inf], 1)[0] == L.ST_ROW_ZERO_MASS


def test_list_status_smallest_code_first():
    assert L.list_status([0, 1], [0, 0], None, 4, 2, 3) == L.ST_Q_BAD_LEN
    assert L.list_status([4, 1], [math.nan, 0], None, 4, 2, 2) == L.ST_Q_BAD_ID
    assert L.list_status([1, 1], [math.nan, 0], None, 4, 2, 2) == L.ST_Q_UNSORTED
    assert L.list_status([0, 1], [math.inf, 0], None, 4, 2, 2) == L.ST_Q_NONFINITE
    assert L.list_status([0, 1], [1, 0], math.nan, 4, 2, 0) == L.ST_OK


def test_distill_of_equal_rows_is_zero():
    x = np.array([0.5, -1.0, 2.0, 0.0])
    loss, grad, *_ = L.distill_row(x, [0, 1, 2, 3], x, 2.0)
    assert abs(loss) < 1e-15 and np.abs(grad).max() < 1e-16
    lse = L.logsumexp(x / 2.0)
    loss, grad, q, p, P, Q = L.distill_row(x, [1, 2], x[[1, 2]], 2.0, lse)
    assert abs(loss) < 1e-15 and np.abs(grad).max() < 1e-15 and abs(P - Q) < 1e-15


def test_distill_without_mass_off_the_list_leaves_the_tail_out():
    x = np.array([0.0, 1.0])
    loss, grad, *_ = L.distill_row(x, [0, 1], [0.0, 0.0], 1.0, lse=2.0)
    assert math.isfinite(loss) and np.isfinite(grad).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temp", [0.7, 2.0])
def test_distill_gradient_against_differences(tail, temp):
    rng = np.random.default_rng(5)
    x, z = rng.normal(0, 2, 12), rng.normal(0, 2, 12)
    ids = np.array([1, 4, 5, 11])
    lse = L.logsumexp(z / temp) if tail else None
    _, grad, *_ = L.distill_row(x, ids, z[ids], temp, lse)
    h = 1e-5  # central differences: off by h^2 times a third derivative below 2, and by 1e-15 / h
    for v in range(12):
        d = np.zeros(12)
        d[v] = h
        up = L.distill_row(x + d, ids, z[ids], temp, lse)[0]
        dn = L.distill_row(x - d, ids, z[ids], temp, lse)[0]
        assert abs((up - dn) / (2 * h) - grad[v]) < 2 * h * h / temp ** 3 + 1e-9
