"""The logit operators as they are used together: raw rows are shaped, then
proposed from, verified, and distilled from."""
import numpy as np
import pytest
import torch

from oracle import logits as L
from vocab_wide_draft_amd import binding as B

from gpu_helpers import dev, to_dev
from test_gpu_distill import check as check_distill
from test_gpu_shape import f32, f64, host64, i32, pack, rows_of
from test_gpu_top_logits import check_rows

pytestmark = pytest.mark.gpu


def test_shape_then_step():
    """Shaped draft and target rows through the fused step: its tokens are
    allowed ones, its argmax that of the shaped rows."""
    rng = np.random.default_rng(31)
    R, V = 3, 4099
    d, t = rows_of(rng, R * 5, V, "f32"), rows_of(rng, R * 6, V, "f32")
    hist = rng.integers(0, V, (R, 64))
    allowed = rng.random((R, V)) < 0.2
    how = dict(history=i32(hist), repetition=f32([1.3] * R), presence=f32([0.5] * R), temperature=f32([0.8] * R),
               mask=i32(pack(allowed)))
    sd = B.shape_logits(to_dev(d, "f32"), 5, mask_row=i32(np.repeat(np.arange(R), 5)), **how)["logits"]
    first = B.propose(sd)["argmax"].view(R, 5)
    st = B.shape_logits(to_dev(t, "f32"), 6, draft=first.contiguous(), mask_row=i32(np.repeat(np.arange(R), 6)), **how)["logits"]
    out = B.fused(sd, st, B.GREEDY, with_q=False)
    assert torch.equal(out["argmax"], first.reshape(-1)) and (out["req_status"] == 0).all()
    assert torch.equal(out["argmax"].long(), sd.argmax(1)) and torch.equal(out["target_argmax"].long(), st.argmax(1))
    for r in range(R):
        assert allowed[r, out["argmax"].view(R, 5)[r].cpu().numpy()].all()
        assert allowed[r, out["target_argmax"].view(R, 6)[r].cpu().numpy()].all()
    # a mask that allows nothing: the step refuses the row
    none = B.shape_logits(to_dev(d, "f32"), 5, mask=i32(np.zeros((1, 129))), mask_row=i32(np.zeros(R * 5)))["logits"]
    assert (B.propose(none)["status"] == L.ST_ROW_ZERO_MASS).all()


@pytest.mark.parametrize("sd,td", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("tail", [True, False])
def test_teacher_rows_to_gradient(sd, td, tail):
    rng = np.random.default_rng(32)
    n, V, k, temp = 10, 6007, 40, 1.5
    t = rows_of(rng, n, V, td, 2.0)
    a = rows_of(rng, n, V, sd, 2.0)
    top = B.top_logits(to_dev(t, td), k, temperature=temp)
    check_rows(t, td, [k] * n, temp, top)
    if not tail:
        top["lse"] = None
    x = to_dev(a, sd).requires_grad_()
    w = f32(rng.random(n))
    loss = B.distill_loss(x, top, temp)
    (loss * w).sum().backward()
    as_list = tuple(None if v is None else v.cpu().numpy() for v in (top["ids"], top["logits"], top["len"], top["lse"]))
    check_distill(a, sd, as_list, temp, w.cpu().numpy(), loss.detach().cpu().numpy(), host64(x.grad))
    step = B.distill_step(to_dev(a, sd), top, w, temp)
    check_distill(a, sd, as_list, temp, w.cpu().numpy(), step["loss"].cpu().numpy(), host64(step["grad"]))


def test_a_training_step_lowers_nothing_it_should_not():
    """One gradient step on the logits themselves moves the student's
    probabilities towards the teacher's: the loss's own first-order change
    is -lr |grad|^2, up to the second-order term lr^2 |grad|^2 / (2 T^2) (the
    Hessian of the loss along any direction is at most 1 / T^2)."""
    rng = np.random.default_rng(33)
    n, V = 4, 2000
    a = rows_of(rng, n, V, "f32", 2.0)
    top = B.top_logits(to_dev(rows_of(rng, n, V, "f32", 2.0), "f32"), 16)
    top["lse"] = None  # a convex loss
    x = to_dev(a, "f32")
    s = B.distill_step(x, top, torch.ones(n, device=dev()))
    g2 = s["grad"].double().square().sum(1)
    after = B.distill(x - 0.5 * s["grad"], top)["loss"].double()
    change = s["loss"].double() - after
    tol = 1e-4  # two losses near 10, each off by less than 2 D + F |loss| < 5e-5
    assert (change >= (0.5 - 0.125) * g2 - tol).all() and (change <= 0.5 * g2 + tol).all()
