"""A teacher's lse that its 24 bits put far below its logits over T: the listed
probabilities sum to more than binary32 holds.  Such a list is refused; what is
not refused has a finite loss and gradient."""
import numpy as np
import pytest
import torch

from oracle import logits as L
from vocab_wide_draft_amd import binding as B
from vocab_wide_draft_amd import workloads as W

from gpu_helpers import dev, to_dev
from test_gpu_shape import f32, i32, rows_of

pytestmark = pytest.mark.gpu


def run(x, tt, w, temp):
    f = B.distill(x, tt, temp)
    g = B.distill_backward(x, tt, f, w, temp)
    s = B.distill_step(x, tt, w, temp)
    return [(f["status"], f["loss"], g), (s["status"], s["loss"], s["grad"])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", [(40, 300), (8, 40003), (130, 40003), (130, 129280)])
@pytest.mark.parametrize("temp", [2.0 ** -30, 2.0 ** -40, 1.3 * 2.0 ** -60, 2.0 ** -100])
def test_teachers_at_low_temperatures(dtype, n, V, temp):
    rng = np.random.default_rng(V + n)
    few = min(n, 40)
    tile = lambda a: np.concatenate([a] * -(-n // few))[:n]
    z, a = tile(rows_of(rng, few, V, dtype)), tile(rows_of(rng, few, V, dtype))
    tt = B.top_logits(to_dev(z, dtype), 30, temperature=temp)
    # the sum in 64 bits from what the call is given, decided far from the border of binary32
    T = float(np.float32(temp))
    with np.errstate(over="ignore"):
        b = np.exp(tt["logits"].double().cpu().numpy() * (1.0 / T) - tt["lse"].double().cpu().numpy()[:, None]).sum(1)
    over, under = b > 1e39, b < 1e38
    assert (over | under).all()
    for status, loss, grad in run(to_dev(a, dtype), tt, torch.ones(n, device=dev()), temp):
        assert status.tolist() == np.where(over, L.ST_Q_NONFINITE, 0).tolist()
        bad = torch.from_numpy(over).to(dev())
        assert not loss[bad].any() and not grad[bad].any()
        # a loss is at most p (z - x) / T with |z - x| < 40, which leaves binary32 only where p does nearly
        assert not loss.isnan().any() and not grad.isnan().any()


@pytest.mark.parametrize("V", [500, 40003])
def test_probabilities_past_binary32(V):
    x = np.zeros((5, V), np.float32)
    x[3, 9] = np.nan
    ids, z = np.tile(np.array([[1, 9]], np.int32), (5, 1)), np.tile(np.array([[200.0, 3.0]], np.float32), (5, 1))
    lse = np.array([100.0, 199.0, -1000.0, 100.0, 100.0], np.float32)  # the sums: e^100, e, past binary64, and e^100 twice
    ln = np.array([2, 2, 2, 2, 0], np.int32)
    for dtype in ("f32", "bf16"):
        a = x if dtype == "f32" else np.where(np.isnan(x), 0x7FC0, W.f32_to_bf16_bits(np.nan_to_num(x))).astype(np.uint16)
        tt = {"ids": i32(ids), "logits": f32(z), "len": i32(ln), "lse": f32(lse)}
        for status, loss, grad in run(to_dev(a, dtype), tt, torch.ones(5, device=dev()), 1.0):
            # the teacher's refusal comes before the student's; an empty list has no sum
            assert status.tolist() == [L.ST_Q_NONFINITE, 0, L.ST_Q_NONFINITE, L.ST_Q_NONFINITE, 0]
            assert not loss[[0, 2, 3, 4]].any() and not grad[[0, 2, 3, 4]].any() and torch.isfinite(grad[1]).all()
