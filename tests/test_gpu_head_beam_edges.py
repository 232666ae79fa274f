"""Cases of the 8-bit head and the beam selection that their kernels' inner limits make: ties in slices of every length,
products of a few steps in tiles of every width, the default number of continuations.  What is compared is exact."""
import numpy as np
import pytest
import torch

from vocab_wide_draft_amd import binding as B

import beam_oracle as O
from head_oracle import KINDS, wide

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V", [(3, 70000), (15, 70000), (32, 70000), (40, 62003)])
def test_ties_in_slices_of_every_length(R, V, dtype):
    """More logits of one value than a slice lists, with few above them or none, the last ones that are selected decided by
    their ids; rows of three tokens over the type's lowest value.  Scores 40 apart, so that no two beams meet but where
    they are meant to."""
    low, g = torch.finfo(dtype).min, torch.Generator().manual_seed(R)
    x = torch.full((R * 2, V), low).to(dtype)
    for r in range(R * 2):
        kind = r % 6
        if kind == 0:
            x[r, torch.randint(0, V, (3,), generator=g)] = torch.tensor([1.0, 2.0, 2.0], dtype=dtype)
        elif kind == 1:
            x[r] = 0.5
        elif kind == 2:
            x[r] = torch.randint(0, 2, (V,), generator=g).to(dtype)
        elif kind == 3:
            x[r] = (torch.randn(V, generator=g) * 0.5).round().to(dtype)
        elif kind == 4:
            x[r, V // 2:] = -1.0
            x[r, V - 5:] = torch.tensor([3.0, 4.0, 5.0, 6.0, 4.0], dtype=dtype)
        else:
            x[r, :] = -0.0
            x[r, ::3] = 0.0
    s = np.tile(np.array([[-1.0, -41.0]], np.float32), (R, 1))
    s[::2] = [[-41.0, -1.0]]
    for n_out in (5, 40):
        got = {k: v.cpu().numpy() for k, v in B.beam_select(wide(x, dev), torch.from_numpy(s).to(dev), n_out).items()}
        parent, token, _, ended, length, status = O.select(x.float().numpy(), s, n_out)
        for name, want in (("status", status), ("len", length), ("parent", parent), ("token", token), ("finished", ended)):
            np.testing.assert_array_equal(got[name], want, name)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("width", [16, 128, 144, 272, 400, 656])
@pytest.mark.parametrize("n", [40, 100, 129, 192, 250])
def test_tiles_of_every_width_and_few_steps(n, width, kind):
    """Whole numbers whose products and sums no step has to round, one to six steps of a tile; 256 tiles of 256 tokens, the
    last one short."""
    V, g = 65500, torch.Generator(device=dev).manual_seed(n + width)
    x = torch.randint(-1, 2, (n, width), generator=g, device=dev).float() * (torch.rand((n, width), generator=g, device=dev) < min(1.0, 100.0 / width))
    w = torch.randint(-2, 3, (V, width), generator=g, device=dev).float()
    sx = 2.0 ** torch.randint(-3, 4, (n, 1), generator=g, device=dev).float().repeat(1, -(-width // 128))
    sw = 2.0 ** torch.randint(-3, 4, (-(-V // 128), 1), generator=g, device=dev).float().repeat(1, -(-width // 128))
    q = [{"values": v.to(torch.float8_e4m3fn), "scales": s.to(KINDS[kind])} for v, s in ((x, sx), (w, sw))]
    want = x @ w.t()  # (whole numbers below 2^24: exact)
    assert want.abs().max() <= 256
    want = want * sx[:, :1] * sw[:, 0].repeat_interleave(128)[:V]
    assert torch.equal(B.block_product(*q, torch.bfloat16).float(), want)
    assert torch.equal(B.block_product(*q, torch.float32), want)


@pytest.mark.parametrize("beams,count", [(1, 2), (32, 64), (45, 90), (46, 89), (64, 64)])
def test_default_count(beams, count):
    """Twice the beams, or what beams * n_out <= 4096 leaves."""
    x = torch.randn((beams, 300), generator=torch.Generator().manual_seed(beams)).to(dev)
    got = B.beam_select(x, torch.zeros((1, beams), device=dev))
    assert got["parent"].shape == (1, count) and int(got["len"][0]) == count


def test_most_beams_over_the_longest_rows():
    """64 beams of 2^20 ids, all masked but some."""
    beams, V, n_out = 64, 1 << 20, 64
    g = torch.Generator().manual_seed(1)
    x = torch.full((beams, V), -np.inf, dtype=torch.bfloat16)
    for r in range(beams):
        x[r, torch.randint(0, V, (2000,), generator=g)] = (torch.randn(2000, generator=g) * 3).to(torch.bfloat16)
    s = (-3 - torch.rand((1, beams), generator=g)).float()
    got = {k: v.cpu().numpy() for k, v in B.beam_select(x.to(dev), s.to(dev), n_out).items()}
    parent, token, _, ended, length, status = O.select(x.float().numpy(), s.numpy(), n_out)
    for name, want in (("status", status), ("len", length), ("parent", parent), ("token", token), ("finished", ended)):
        np.testing.assert_array_equal(got[name], want, name)


def test_a_transposed_head_of_another_size_is_refused_at_once():
    w = B.quantize_blocks(torch.ones((200, 64), device=dev), 128)
    x = torch.ones((3, 64), device=dev, requires_grad=True)
    for t in (B.quantize_blocks(torch.ones((64, 176), device=dev), 128), B.quantize_blocks(torch.ones((48, 200), device=dev), 128)):
        with pytest.raises(ValueError, match="transposed"):
            B.head_logits(x, {"weight": w, "transposed": t})
    assert B.head_logits(x, {"weight": w, "transposed": B.transpose_blocks(w, 64)}).shape == (3, 200)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("width", [16, 400])
@pytest.mark.parametrize("n", [193, 257, 264, 330, 400, 450, 520, 600, 700])
def test_a_narrower_last_tile(n, width, kind):
    test_tiles_of_every_width_and_few_steps(n, width, kind)
