"""The distillation where its last term is left out (its gradient then has
the softmax times b = sum p, which is not one).

Tolerances, counted before the first run, with F = 2^-24, t the distance from
the row's maximum over T and D = F (3 E[t] + 162) for a sum of exponentials
(see test_gpu_distill): q_v is off by D + F (3 t_v + 6) of itself and is scaled
by b; the products and p add 4 F of b q + p; the hardware exponential's
underflow 2^-126 b; bf16 half a step, 2^-8, of the result.  Over a whole row
these errors add up to at most (b (D + F (3 E[t] + 10)) + 4 F b + 2^-8 sum |g|)."""
import numpy as np
import pytest
import torch

from oracle import logits as L
from vocab_wide_draft_amd import binding as B
from vocab_wide_draft_amd import workloads as W

from gpu_helpers import to_dev
from test_gpu_distill import teacher
from test_gpu_shape import f32, f64, host64

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
SIZES = [(3, 60), (8, 60), (3, 9000), (3, 40003), (8, 40003), (8, 129280), (130, 40003), (130, 70001), (3, 129280), (130, 129280)]


def both(a, dtype, t, temp, weight):
    x, tt, w = to_dev(a, dtype), teacher(t), f32(weight)
    f = B.distill(x, tt, temp)
    g = B.distill_backward(x, tt, f, w, temp)
    s = B.distill_step(x, tt, w, temp)
    assert not f["status"].any() and not s["status"].any()
    return (f["loss"], g), (s["loss"], s["grad"])


def tiled(n, few, *arrays):
    rep = -(-n // few)
    return [None if v is None else np.concatenate([v] * rep)[:n] for v in arrays]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", SIZES)
@pytest.mark.parametrize("how", ["no logit off the list", "probabilities above one"])
def test_gradient_without_the_last_term(how, n, V, dtype):
    rng = np.random.default_rng(V + n)
    k, temp, few = 12, 1.5, 3
    x = (rng.standard_normal((few, V)) * 2).astype(np.float32)
    z = rng.normal(0, 2, (few, k)).astype(np.float32)
    ids = np.stack([np.sort(rng.permutation(V)[:k]) for _ in range(few)]).astype(np.int32)
    true = np.array([L.logsumexp(z[r].astype(np.float64) / temp) for r in range(few)])
    if how == "no logit off the list":
        only = np.full_like(x, -np.inf)
        for r in range(few):
            only[r, ids[r]] = x[r, ids[r]]
        x, lse = only, (true + [0.5, 1.5, 3.0]).astype(np.float32)
    else:
        lse = (true - [0.01, 0.4, 1.0]).astype(np.float32)
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    weight = np.array([1.0, -0.7, 0.3], np.float32)
    ln = np.full(few, k, np.int32)
    big = tiled(n, few, a, ids, z, ln, lse, weight)
    for loss, grad in both(big[0], dtype, tuple(big[1:5]), temp, big[5]):
        got = host64(grad[:few])
        for r in range(few):
            row = f64(a[r], dtype)
            wl, _, q, p, P, Q = L.distill_row(row, ids[r], z[r], temp, lse[r])
            b, w = p.sum(), float(weight[r]) / temp
            assert P == 0 and abs(b - 1) > 0.005
            with np.errstate(invalid="ignore"):
                t = np.where(row > -np.inf, (row.max() - row) / temp, 0.0)
            D = F * (3 * (q * t).sum() + 162)
            assert abs(float(loss[r]) - wl) <= 2 * D * max(1.0, b) + F * abs(wl) + 1e-12
            want = w * (b * q - p)
            tol = abs(w) * (b * (q * (D + F * (3 * t + 6)) + 2.0 ** -126) + 4 * F * (b * q + p)) + 2.0 ** -133
            total = abs(w) * b * (D + F * (3 * (q * t).sum() + 14)) + V * 2.0 ** -126
            if dtype == "bf16":
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
                total = total * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want).sum()
            bad = np.abs(got[r] - want) > tol
            assert not bad.any(), (r, got[r][bad][:4], want[bad][:4], tol[bad][:4])
            assert abs(got[r].sum()) <= total, (r, got[r].sum(), total)
        assert torch.equal(grad[few * (n // few - 1):few * (n // few)].float(), grad[:few].float())
