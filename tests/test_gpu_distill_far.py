"""The distillation of student rows far from zero: all, or nearly all, of a
row at the lowest value of its type, as masks leave it, and large logits of
either sign.  Only differences of logits matter to the loss, so the bounds are
those of test_gpu_distill."""
import numpy as np
import pytest

from oracle import logits as L
from vocab_wide_draft_amd import workloads as W

from gpu_helpers import to_dev
from test_gpu_distill import check
from test_gpu_distill_limits import SIZES, both, tiled
from test_gpu_shape import host64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", SIZES)
def test_rows_far_from_zero(tail, n, V, dtype):
    rng = np.random.default_rng(V + 2 * n)
    k, few = 12, 8
    low = np.float32(-3.3895313892515355e38) if dtype == "bf16" else np.finfo(np.float32).min
    x = np.empty((few, V), np.float32)
    x[0] = low                                             # everything masked by the type's lowest value
    x[1] = np.where(rng.random(V) < 0.9, low, low * 0.5)   # nearly so
    x[2], x[3], x[4] = 1e12, 1e20, -1e20
    x[5] = 1e6 + 4096 * rng.integers(0, 2, V)              # two values (a step of bf16 there is 4,096)
    x[6] = rng.standard_normal(V)
    x[6, rng.random(V) < 0.5] = low
    x[7] = -3e4 + rng.standard_normal(V)
    z = rng.normal(0, 2, (few, k)).astype(np.float32)
    ids = np.stack([np.sort(rng.permutation(V)[:k]) for _ in range(few)]).astype(np.int32)
    x[6, ids[6]] = 1.0                                     # (a listed logit at the lowest value makes the loss as large)
    x[1, ids[1]] = low * 0.5
    lse = np.array([L.logsumexp(z[r].astype(np.float64)) + 0.3 for r in range(few)], np.float32) if tail else None
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    weight = rng.normal(0, 1, few).astype(np.float32)
    big = tiled(n, few, a, ids, z, np.full(few, k, np.int32), lse, weight)
    rows = range(min(n, few))
    for loss, grad in both(big[0], dtype, tuple(big[1:5]), 1.0, big[5]):
        check(big[0], dtype, tuple(big[1:5]), 1.0, big[5], loss.cpu().numpy(), host64(grad), rows)


@pytest.mark.parametrize("V", [9000, 40003])
def test_listed_logits_at_the_lowest_value(V):
    """Their tokens cost the loss what their probability times that value is, and no more."""
    rng = np.random.default_rng(V)
    x = rng.standard_normal((2, V)).astype(np.float32)
    ids = np.tile(np.array([[1, 700, V - 1]], np.int32), (2, 1))
    z = np.array([[2.0, 1.0, -1.0]] * 2, np.float32)
    x[0, 700] = np.finfo(np.float32).min
    x[1, [1, 700]] = np.finfo(np.float32).min
    t = (ids, z, np.full(2, 3, np.int32), None)
    for loss, grad in both(x, "f32", t, 1.0, np.ones(2, np.float32)):
        check(x, "f32", t, 1.0, np.ones(2), loss.cpu().numpy(), host64(grad))
