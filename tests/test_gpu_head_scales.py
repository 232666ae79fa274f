"""Products of quantised matrices whose scales lie at the ends of binary32, with results within its range.  Tolerances:
test_gpu_head's, and for each block of columns what the interface says of numbers below 2^-126: a product of two scales is off
by up to half of binary32's last place, 2^-150, which the block's sum (128 products of up to 448^2) multiplies, and a sum may
count as zero."""
import pytest
import torch

from vocab_wide_draft_amd import binding as B

from head_oracle import KINDS

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")

# rows and matrices for each of the kernels: straight from memory, staged, tiles of one to four 64s
SIZES = [(1, 300, 528), (20, 1000, 272), (3, 129280, 1024), (20, 129280, 1024), (40, 700, 400), (100, 700, 400), (250, 700, 400), (264, 65500, 272), (5, 40, 20000)]


def _values(n, cols, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn((n, cols), generator=g, device=dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)


def _scales(shape, low, high, kind, seed):
    """Powers of two between 2^low and 2^high, times numbers in [1, 2) where scales are float."""
    g = torch.Generator(device=dev).manual_seed(seed)
    e = torch.randint(low, high + 1, shape, generator=g, device=dev).double()
    m = 1.0 + torch.rand(shape, generator=g, device=dev).double() if kind == "f32" else 1.0
    return (2.0 ** e * m).float().to(KINDS[kind])


def _worth(q, rows):
    v, s = q["values"].double(), q["scales"].float().double()
    return v * s.repeat_interleave(rows, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low,high", [((-126, -120), (-20, -19)), ((-76, -70), (-70, -66)), ((-24, -20), (-126, -120)),
                                      ((100, 119), (-126, -124)), ((-126, -124), (100, 119)), ((-20, -10), (20, 30))])
@pytest.mark.parametrize("n,V,width", SIZES)
def test_products_of_far_scales(n, V, width, low, high, out, kind):
    blocks = -(-width // 128)
    x = {"values": _values(n, width, 1), "scales": _scales((n, blocks), *low, kind, 2)}
    w = {"values": _values(V, width, 3), "scales": _scales((-(-V // 128), blocks), *high, kind, 4)}
    got = B.block_product(x, w, out).double()
    X, W = _worth(x, 1), _worth(w, 128)
    want, size = X @ W.t(), X.abs() @ W.abs().t()
    tol = size * ((width + 2 * (width // 128 + 1) + 4) * 2.0 ** -24) + blocks * (128 * 448.0 ** 2 * 2.0 ** -150 + 2.0 ** -126)
    if out == torch.bfloat16:
        tol = tol + size * (7 * 2.0 ** -13)
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    off = (got - want).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), float((off / tol).max())

