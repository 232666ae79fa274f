"""What the operators on logit rows write in place counts as written for
torch: a backward pass that needs the overwritten values refuses to run."""
import numpy as np
import pytest
import torch

from vocab_wide_draft_amd import binding as B

from gpu_helpers import dev, to_dev
from test_gpu_distill import lists, teacher
from test_gpu_shape import f32, f64, rows_of

pytestmark = pytest.mark.gpu
WRITES = ["shape", "step", "backward"]


def write(how, x, tt, w, out):
    if how == "shape":
        return B.shape_logits(x, temperature=w, out=out)["logits"]
    if how == "step":
        return B.distill_step(x, tt, w, out=out)["grad"]
    return B.distill_backward(x, tt, B.distill(x, tt), w, out=out)


@pytest.mark.parametrize("where", ["the rows", "a view of them", "other memory"])
@pytest.mark.parametrize("how", WRITES)
def test_writes_are_seen_by_autograd(how, where):
    rng = np.random.default_rng(51)
    n, V = 4, 2000
    a = rows_of(rng, n, V, "f32", 2.0)
    tt, w = teacher(lists(rng, f64(a, "f32"), 20, 1.0, True)), f32(np.full(n, 2.0))
    z = to_dev(a, "f32").requires_grad_()
    student = z * 1.0
    kept = B.distill_loss(student, tt)
    if where == "other memory":
        out = torch.empty_like(student)
        v = out._version
        got = write(how, student.detach(), tt, w, out)
        assert got.data_ptr() == out.data_ptr() and out._version > v
        (g,) = torch.autograd.grad(kept.sum(), z)  # the student rows were left alone
        want = B.distill_backward(to_dev(a, "f32"), tt, B.distill(to_dev(a, "f32"), tt), torch.ones(n, device=dev()))
        assert torch.equal(g, want)
        return
    out = student.detach() if where == "the rows" else student.detach()[:, :V]
    write(how, out, tt, w, out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.sum().backward()


@pytest.mark.parametrize("how", WRITES)
def test_writes_without_autograd(how):
    """Inference tensors keep no versions; results are those of memory apart."""
    rng = np.random.default_rng(52)
    n, V = 3, 1000
    a = rows_of(rng, n, V, "bf16", 2.0)
    tt, w = teacher(lists(rng, f64(a, "bf16"), 20, 1.0, True)), f32(np.full(n, 2.0))
    want = write(how, to_dev(a, "bf16"), tt, w, None)
    with torch.inference_mode():
        x = to_dev(a, "bf16")
        got = write(how, x, tt, w, x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
