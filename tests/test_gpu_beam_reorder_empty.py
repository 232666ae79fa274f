"""Reordering where some states, or all, hold nothing (caches before the first position): parents and lengths are looked at
all the same."""
import pytest
import torch

from vocab_wide_draft_amd import binding as B

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
OK, BAD_PARENT, BAD_LENGTH = 0, 24, 25


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


PARENT = [[1, 0], [0, 0], [2, 0], [1, -1], [1, 1], [-2, 0]]


@pytest.mark.parametrize("place", [True, False])
def test_no_positions_yet(place):
    x = [torch.zeros((6, 2, 0, 8), device=dev) for _ in range(3)]
    out = None if place else [t.clone() for t in x]
    assert B.beam_reorder(x, _i32(PARENT), out=out)["status"].tolist() == [OK, OK, BAD_PARENT, OK, OK, BAD_PARENT]
    got = B.beam_reorder(x, _i32(PARENT), _i32([0, 0, 0, 1, -1, 5]), out=out)
    assert got["status"].tolist() == [OK, OK, BAD_PARENT, BAD_LENGTH, BAD_LENGTH, BAD_PARENT]
    with pytest.raises(ValueError):
        B.beam_reorder(x, _i32(PARENT).long())
    with pytest.raises(ValueError):
        B.beam_reorder(x, _i32(PARENT), torch.zeros(6, dtype=torch.int64, device=dev))


def test_an_empty_state_among_others():
    """A request whose length passes what one state has is left as it is in all of them."""
    full = torch.arange(6 * 2 * 4, device=dev).view(6, 2, 4).contiguous()
    for empty, lengths, want in ((torch.zeros((6, 2, 0, 8), device=dev), [0, 0, 0, 1, 4, 0], [0, 0, 24, 25, 25, 24]),
                                 (torch.zeros((6, 2, 3, 0), device=dev), [3, 2, 3, 4, 0, 3], [0, 0, 24, 25, 0, 24])):
        x = full.clone()
        got = B.beam_reorder([empty, x], _i32(PARENT), _i32(lengths))
        assert got["status"].tolist() == want
        ref = full.clone()
        for r, (n, st) in enumerate(zip(lengths, want)):
            if st == 0:
                for b, p in enumerate(PARENT[r]):
                    if p >= 0:
                        ref[r, b, :n] = full[r, p, :n]
        assert torch.equal(x, ref)


def test_nothing_to_reorder():
    assert B.beam_reorder([torch.zeros((0, 2, 4), device=dev)], torch.zeros((0, 2), dtype=torch.int32, device=dev))["status"].shape == (0,)
