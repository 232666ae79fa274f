"""Top logits of rows of the largest vocabulary (128 slices a row), with lists
whose candidates fill the selection's room and, in some rows, pass it."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, to_dev
from test_gpu_shape import rows_of
from test_gpu_top_logits import check_rows
from vocab_wide_draft_amd import binding as B
from vocab_wide_draft_amd import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(1 << 20, 1024), (1 << 20, 256), (1 << 20, 1), ((1 << 20) - 3, 1024), (524288, 1024)])
def test_top_of_the_longest_rows(dtype, V, k):
    rng = np.random.default_rng(V + k)
    a = rows_of(rng, 6, V, dtype)
    g = B.top_logits(to_dev(a, dtype), k, temperature=1.2)
    check_rows(a, dtype, [k] * 6, 1.2, g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_top_where_candidates_pass_the_room(dtype):
    """The sampled logits 1 lower than the rest: the threshold lets several times too many through."""
    rng = np.random.default_rng(3)
    V = 1 << 20
    x = (rng.standard_normal((2, V)) * 3).astype(np.float32)
    for c in range(64):
        x[:, c * (V // 64):c * (V // 64) + 32] -= 1.0
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    ks = np.array([1024, 700], np.int32)
    g = B.top_logits(to_dev(a, dtype), 1024, topk=torch.from_numpy(ks).to(dev()))
    check_rows(a, dtype, ks, 1.0, g)
