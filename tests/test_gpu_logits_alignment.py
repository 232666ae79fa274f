"""Rows that do not start 16-byte aligned: refused, with the reason, by every
operator on logit rows; the same logits as the first columns of a wider tensor
are taken."""
import numpy as np
import pytest
import torch

from vocab_wide_draft_amd import binding as B

from gpu_helpers import dev
from test_gpu_distill import lists, teacher

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_rows(dtype):
    rng = np.random.default_rng(61)
    n, V = 3, 20003
    a = rng.standard_normal((n, V)).astype(np.float32)
    x = torch.from_numpy(a).to(dev()).to(dtype)
    t = teacher(lists(rng, a.astype(np.float64), 9, 1.0, True, ragged=False))
    w = torch.ones(n, device=dev())
    rows = torch.empty((n, -(-V // 8) * 8), dtype=dtype, device=dev())[:, :V].copy_(x)
    stats = B.distill(rows, t)
    calls = [lambda y: B.shape_logits(y)["logits"], lambda y: B.top_logits(y, 5)["lse"], lambda y: B.distill(y, t)["loss"],
             lambda y: B.distill_step(y, t, w)["grad"], lambda y: B.distill_backward(y, t, stats, w), lambda y: B.distill_loss(y, t),
             lambda y: B.shape_logits(rows, out=y)["logits"], lambda y: B.distill_step(rows, t, w, out=y)["grad"]]
    for call in calls:
        with pytest.raises(B.DsparkError, match="16-byte aligned"):
            call(x)
    assert torch.equal(calls[0](rows), x)
    one = rows[:, 1:]  # aligned in its stride, not where it starts
    with pytest.raises(B.DsparkError, match="16-byte aligned"):
        B.top_logits(one, 5)
    room = torch.empty((n, -(-V // 8) * 8), dtype=dtype, device=dev())[:, :V]
    for call in calls:
        assert torch.isfinite(call(rows if call in calls[:6] else room)).all()
