"""The log-sum-exp of top logits far from zero: low temperatures and large
logits, where a maximum over the temperature has few or no bits behind the
point.

Bound, counted before the first run, with t = (max - x) / T and F = 2^-24.
Near zero an exponent is fma(x, c, -K), K = m c rounded: the fused
multiply-add rounds once (t F, and F times the residual of K, 2 at most), c is
off by F of itself (t F more, as what it does to the maximum is put back).
Far from zero it is (x - m) c: three roundings, 3 t F.  The hardware
exponential is off by 2 F, a thread and its wave add at most 38 binary32
values, the result is rounded once: F of |lse|, which far from zero is nearly
all of it."""
import numpy as np
import pytest
import torch

from oracle import logits as L
from vocab_wide_draft_amd import binding as B
from vocab_wide_draft_amd import workloads as W

from gpu_helpers import dev, to_dev
from test_gpu_shape import f64, rows_of

pytestmark = pytest.mark.gpu
F = 2.0 ** -24


def check_lse(a, dtype, temp, g, rows):
    lse, st = g["lse"].cpu().numpy(), g["status"].cpu().numpy()
    for r in rows:
        x = f64(a[r], dtype)
        t = (x.max() - x) / temp
        w = np.exp(-t)
        part = np.where(w > 0, w * (3 * np.where(w > 0, t, 0.0) + 44), 0.0).sum() / w.sum()
        want = x.max() / temp + np.log(w.sum())
        assert st[r] == 0 and abs(float(lse[r]) - want) <= F * (part + abs(want)) * 1.001, (r, lse[r], want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", [(4, 300), (4, 20003), (540, 8000)])
@pytest.mark.parametrize("temp", [2.0 ** -22, 2.0 ** -24, 2.0 ** -26, 2.0 ** -28, 1.25 * 2.0 ** -30, 2.0 ** -32, 2.0 ** -40,
                                  2.0 ** -60, 1.5 * 2.0 ** -61, 2.0 ** -90])
def test_lse_at_low_temperatures(dtype, n, V, temp):
    rng = np.random.default_rng(V + 5)
    a = rows_of(rng, 4, V, dtype)
    g = B.top_logits(to_dev(np.tile(a, (n // 4, 1)), dtype), 20, temperature=temp)
    check_lse(a, dtype, temp, g, range(4))
    assert all(torch.equal(g["lse"][i::4], g["lse"][i].expand(n // 4)) for i in range(4))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", [(8, 300), (8, 20003), (544, 8000)])
@pytest.mark.parametrize("size", [4.6e7, 1e9, 3.3e9, 1e10, 1e20, 1e28, 3e38])
def test_lse_of_large_logits(dtype, n, V, size):
    """Rows of one size and either sign, around 2^26 / log2 e = 4.65e7 among them, spread over a few steps of
    their type or as a whole, and rows of which a part is small."""
    rng = np.random.default_rng(V + 6)
    x = np.empty((8, V))
    step = 2.0 ** (-8 if dtype == "bf16" else -23)
    x[0] = size * (1 - step * rng.integers(0, 4, V))
    x[1] = -size * (1 + step * rng.integers(0, 4, V))
    x[2] = size * rng.uniform(-1, 1, V)
    x[3] = size
    x[4] = -size
    x[5] = np.where(np.arange(V) < V // 2, rng.normal(0, 2, V), -size)
    x[6] = np.where(np.arange(V) < V // 2, -size, -size * 0.75)
    x[7] = np.where(rng.random(V) < 0.01, size * 1.01, rng.normal(0, 2, V))
    x = x.astype(np.float32)
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    g = B.top_logits(to_dev(np.tile(a, (n // 8, 1)), dtype), 20)
    check_lse(a, dtype, 1.0, g, range(8))
    for r in range(8):
        s, ids, z, _ = L.top_row(f64(a[r], dtype), 20)
        assert g["ids"][r, :len(ids)].tolist() == ids.tolist() and g["logits"][r, :len(ids)].tolist() == z.tolist()


def test_lse_past_binary32():
    """A log-sum-exp that binary32 cannot hold is infinite, as its rounding is; a list with it is refused."""
    x = torch.zeros((2, 300), device=dev())
    x[0, 5], x[1] = 1e38, -1e38
    g = B.top_logits(x, 3, temperature=2.0 ** -10)
    assert g["status"].tolist() == [0, 0] and g["lse"].tolist() == [float("inf"), -float("inf")]
    assert B.distill(torch.zeros((2, 300), device=dev()), g, 2.0 ** -10)["status"].tolist() == [L.ST_Q_NONFINITE] * 2
