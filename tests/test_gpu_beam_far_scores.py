"""Beam selection where scores leave binary32: beams whose scores, or rows whose masked logits, are the types' lowest
values, so that their sum is finite in binary64 and rounds to -inf.  Such a candidate comes after those above it and
before an empty slot.  Everything compared is exact but the scores, whose tolerance is test_gpu_beam's."""
import numpy as np
import pytest
import torch

from vocab_wide_draft_amd import binding as B

import beam_oracle as O
from head_oracle import wide

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
LOW = np.finfo(np.float32).min


def _same(x, s, n_out):
    got = {k: v.cpu().numpy() for k, v in B.beam_select(wide(x, dev), torch.from_numpy(s).to(dev), n_out).items()}
    parent, token, score, ended, length, status = O.select(x.float().numpy(), s, n_out)
    for name, want in (("status", status), ("len", length), ("parent", parent), ("token", token), ("finished", ended)):
        np.testing.assert_array_equal(got[name], want, name)
    with np.errstate(over="ignore"):
        want = score.astype(np.float32)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got["score"][~fine], want[~fine])
    off = np.abs(got["score"][fine].astype(np.float64) - score[fine])
    assert (off <= 2e-6 + np.abs(score[fine]) * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,beams,V,n_out,few", [
    (1, 8, 20003, 20, 3),      # lists by the slice, fewer of them with a finite best than are selected
    (3, 16, 9000, 16, 3),
    (1, 32, 20003, 64, 40),
    (2, 4, 3000, 8, 3),        # few lists: the threads' best
    (1, 3, 5, 15, 2),          # all of them selected, those that round to -inf too
    (1, 8, 20003, 20, 1),      # equal logits in number: the lists of every beam, merged
    (1, 64, 300, 64, 1)])
def test_scores_below_binary32(R, beams, V, n_out, few, dtype):
    """Rows masked with the type's lowest value but for a few neighbouring ids; all beams but the first at float32's."""
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(V + beams)
    x = torch.full((R * beams, V), low).to(dtype)
    for r in range(R * beams):
        at = int(torch.randint(0, V - few + 1, (1,), generator=g))
        x[r, at:at + few] = (torch.randn(few, generator=g) * 2).to(dtype)
    s = np.full((R, beams), LOW, np.float32)
    s[:, 0] = -1.0
    _same(x, s, n_out)
    s[:, 0] = LOW       # none of them above it
    _same(x, s, n_out)
    s[:, -1] = -2.0     # the last one is the only one
    s[:, ::2] = -np.inf
    _same(x, s, n_out)
