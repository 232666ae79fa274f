"""Beam selection against the plain form in extended precision, and the reordering of states against indexing.

Tolerances.  Whole outputs are equal.  A score is s + (x - lse) in binary64 with the log-sum-exp from binary32
exponentials, off by at most 2e-6 (each exponential by (|t| 0.7 + 2) 2^-24 of itself, t its exponent in base 2, whose
weighted mean is below 18; a term is in twelve binary32 sums), rounded to binary32: half a step, 2^-24 of itself."""
import numpy as np
import pytest
import torch

from vocab_wide_draft_amd import binding as B

import beam_oracle as O
from head_oracle import wide

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
NINF = -np.inf


def _run(x, scores, n_out, finished=None, end_token=-1):
    """Through the library; x: a CPU tensor [rows, V]."""
    f = None if finished is None else torch.from_numpy(np.asarray(finished, np.int32)).to(dev)
    s = torch.from_numpy(np.ascontiguousarray(scores, np.float32)).to(dev)
    return {k: v.cpu().numpy() for k, v in B.beam_select(wide(x, dev), s, n_out, finished=f, end_token=end_token).items()}


def _same(got, x, scores, n_out, finished=None, end_token=-1):
    scores = np.asarray(scores, np.float32)
    parent, token, score, ended, length, status = O.select(x.float().numpy(), scores, n_out, finished, end_token)
    np.testing.assert_array_equal(got["status"], status)
    np.testing.assert_array_equal(got["len"], length)
    np.testing.assert_array_equal(got["parent"], parent)
    np.testing.assert_array_equal(got["token"], token)
    np.testing.assert_array_equal(got["finished"], ended)
    fine = np.isfinite(score)
    np.testing.assert_array_equal(got["score"][~fine], score[~fine].astype(np.float32))
    tol = 2e-6 + np.abs(score[fine]) * 2.0 ** -24
    assert (np.abs(got["score"][fine].astype(np.float64) - score[fine].astype(np.float64)) <= tol).all()


def _rows(n, V, dtype, seed, scale=3.0):
    return (torch.randn((n, V), generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _scores(R, beams, seed):
    return -np.sort(np.abs(np.random.default_rng(seed).standard_normal((R, beams))) * 5 + 3, 1).astype(np.float32)


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,beams,V,n_out", [(1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 6), (3, 2, 1000, 4), (1, 4, 2048, 8), (1, 4, 2049, 8),
                                             (2, 5, 8193, 10), (7, 8, 20003, 16), (1, 4, 129280, 8), (1, 64, 3000, 64),
                                             (2, 32, 5000, 128), (130, 2, 9000, 4), (1, 1, 70000, 128), (40, 16, 8192, 32)])
def test_select(R, beams, V, n_out, dtype):
    x, s = _rows(R * beams, V, dtype, V + beams), _scores(R, beams, V)
    _same(_run(x, s, n_out), x, s, n_out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,beams,V,n_out", [(3, 4, 50, 8), (6, 8, 3000, 16), (2, 6, 20003, 12), (100, 4, 9000, 8)])
def test_masks_ended_and_empty_beams(R, beams, V, n_out, dtype):
    rng = np.random.default_rng(V)
    x, s = _rows(R * beams, V, dtype, V), _scores(R, beams, V)
    for r in range(R * beams):
        kind = r % 5
        if kind == 1:
            x[r, torch.from_numpy(rng.random(V) < 0.9)] = NINF
        elif kind == 2:
            x[r] = NINF
        elif kind == 3:
            x[r, torch.from_numpy(rng.permutation(V)[3:])] = NINF  # three tokens
        elif kind == 4:
            x[r, torch.from_numpy(rng.random(V) < 0.5)] = torch.finfo(dtype).min
    finished = (rng.random((R, beams)) < 0.3).astype(np.int32) * 7
    s[rng.random((R, beams)) < 0.2] = NINF
    s[0] = NINF           # no beam at all
    x.view(R, beams, V)[1][torch.from_numpy(np.isneginf(s[1]) | (finished[1] != 0))] = float("nan")  # rows that are not read
    got = _run(x, s, n_out, finished, 2)
    assert got["len"][0] == 0
    _same(got, x, s, n_out, finished, 2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [9, 2048, 8192, 30000])
def test_equal_logits(V, dtype):
    """Rows of one value, of three values, and alike beams: lower beams, then lower tokens."""
    x = torch.zeros((12, V), dtype=dtype)
    x[1] = -5.0
    x[2:4] = (torch.arange(V) % 3).to(dtype)
    x[4:6] = _rows(1, V, dtype, 1)
    x[6, ::2], x[6, 1::2] = 0.0, -0.0
    x[7] = -0.0
    x[8:12] = _rows(4, V, dtype, 2).mul(0.3).round()
    s = np.array([[-1, -1, -2, -2], [-3, -3, -0.5, -0.5], [-1, -1, -1, -1]], np.float32)
    for n_out in (1, 8, 100):
        _same(_run(x, s, n_out), x, s, n_out)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_that_lie_close_together(dtype):
    """Candidates of two beams nearer to each other than binary32 exponentials tell: the order of the exact scores."""
    V, n, found = 5000, 60, 0
    x = _rows(2 * n, V, dtype, 5, 2.0)
    s = np.zeros((n, 2), np.float32)
    f = x.float().numpy()
    for r in range(n):
        a, b = f[2 * r], f[2 * r + 1]
        i, j = r % 3, (r // 3) % 3  # which of their best meet
        want = (np.sort(a)[-1 - i] - O.lse(a)) - (np.sort(b)[-1 - j] - O.lse(b))
        s[r, 1] = np.float32(want) + np.float32((r % 7 - 3) * 1e-8)
        gap = float(s[r, 1] - want)
        found += abs(gap) < 4e-7
    assert found > n // 2
    for n_out in (1, 2, 3, 6):
        _same(_run(x, s, n_out), x, s, n_out)


@pytest.mark.parametrize("dtype", DTYPES)
def test_refused_requests(dtype):
    x, s = _rows(6 * 3, 700, dtype, 1), _scores(6, 3, 1)
    x[0, 5] = float("nan")
    x[4, 699] = float("inf")
    x[5, 1] = float("nan")
    s[2, 1] = np.nan
    s[3, 0] = np.inf
    x[12, 3] = float("inf")
    got = _run(x, s, 6)
    assert got["status"].tolist() == [1, 1, 23, 23, 2, 0]
    _same(got, x, s, 6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale,shift", [(0.0, 0.0), (1e-3, 0.0), (30.0, 0.0), (1.0, 1e4), (1.0, -3e5), (1e6, 1e9), (1e36, 0.0)])
def test_far_logits(scale, shift, dtype):
    x = (_rows(8, 3000, torch.float32, 3, 1.0) * scale + shift).to(dtype)
    s = _scores(2, 4, 3)
    got = _run(x, s, 8)
    parent, token, score, *_ = O.select(x.float().numpy(), s, 8)
    size = float(x.float().abs().max())
    if size < 1e6:
        _same(got, x, s, 8)
    else:  # (scores beyond 1e6 round to binary64 of themselves: only their values are compared)
        np.testing.assert_allclose(got["score"], score.astype(np.float64), rtol=2.0 ** -23, atol=2e-6 + size * 2.0 ** -50)


def test_longest_rows():
    V = 1 << 20
    for dtype in DTYPES:
        x, s = _rows(3, V, dtype, 9), _scores(1, 3, 9)
        x[1, V - 1] = 20.0
        for n_out in (6, 128):
            _same(_run(x, s, n_out), x, s, n_out)


def test_default_count_and_no_rows():
    x, s = _rows(6, 100, torch.float32, 1), _scores(2, 3, 1)
    got = B.beam_select(wide(x, dev), torch.from_numpy(s).to(dev))
    assert got["parent"].shape == (2, 6)
    got = B.beam_select(torch.empty((0, 100), device=dev), torch.empty((0, 3), device=dev), 6)
    assert got["parent"].shape == (0, 6) and got["len"].shape == (0,)


def test_a_workspace_of_more_rows_serves_fewer():
    lib = B.load_library()
    for V in (1000, 9000, 129280, 262144, 1 << 20):
        big = [lib.dspark_beam_select_workspace(n, V, 8) for n in (1, 3, 8, 30, 31, 32, 33, 60, 64, 200, 511, 512, 600, 3000)]
        assert big == sorted(big)


def test_select_on_streams_and_in_graphs():
    """Two calls at once on streams of their own, and a captured call replayed with other rows and scores."""
    sets = [(wide(_rows(8, 20000, torch.bfloat16, k), dev), torch.from_numpy(_scores(2, 4, k)).to(dev)) for k in (1, 2)]
    want = [B.beam_select(*t, 8) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, t in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append([B.beam_select(*t, 8) for _ in range(4)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(o[k], w[k]) for o in g for k in w)
    x, s = sets[0][0].clone(), sets[0][1].clone()
    x = wide(x.cpu(), dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = B.beam_select(x, s, 8)
    for k in (1, 0, 1):
        x.copy_(sets[k][0])
        s.copy_(sets[k][1])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[k][n]) for n in out)
        B.beam_select(*sets[0], 8)


def test_select_refusals():
    x, s = torch.zeros((6, 104), device=dev), torch.zeros((2, 3), device=dev)
    for bad in (dict(n_out=0), dict(n_out=129), dict(n_out=4, end_token=104), dict(n_out=4, end_token=-2),
                dict(n_out=4, finished=torch.zeros((2, 3), dtype=torch.int32, device=dev))):
        with pytest.raises(B.DsparkError):
            B.beam_select(x, s, **bad)
    with pytest.raises(ValueError):
        B.beam_select(x, torch.zeros((3, 3), device=dev), 4)
    with pytest.raises(ValueError):
        B.beam_select(x, s.double(), 4)
    with pytest.raises(ValueError):
        B.beam_select(x, s, 4, finished=torch.zeros((3, 2), dtype=torch.int32, device=dev), end_token=1)
    with pytest.raises(B.DsparkError):
        B.beam_select(torch.zeros((128, 104), device=dev), torch.zeros((2, 64), device=dev), 128)  # more than 4,096 in a request


# ------------------------------------------------------------ reordering
def _parents(R, beams, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, beams, (R, beams), generator=g, dtype=torch.int32)
    p[torch.rand((R, beams), generator=g) < 0.1] = -1
    if R > 1:
        p[0] = torch.arange(beams, dtype=torch.int32).flip(0)   # everybody moves
        p[1] = torch.arange(beams, dtype=torch.int32)           # nobody does
    return p


def _want(x, parent, length, axis, into):
    """By indexing, on the CPU."""
    out = into.clone()
    for r in range(parent.shape[0]):
        for b in range(parent.shape[1]):
            p = int(parent[r, b])
            if p < 0:
                continue
            if length is None or x.dim() <= axis:
                out[r, b] = x[r, p]
            else:
                at = (slice(None),) * (axis - 2) + (slice(0, int(length[r])),)
                out[r, b][at] = x[r, p][at]
    return out


def _state(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn(shape, generator=g).to(dtype)
    return torch.randint(0, 120, shape, generator=g).to(dtype)


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float64])
@pytest.mark.parametrize("beams", [1, 2, 5, 8, 13, 16, 17, 32, 33, 64])
def test_reorder(beams, dtype, place):
    R = 3
    shapes = [(R, beams, 37, 24), (R, beams, 37, 2, 8), (R, beams, 41, 5), (R, beams, 40), (R, beams, 38, 1, 3)]
    states = [_state(s, dtype, i) for i, s in enumerate(shapes)]
    parent = _parents(R, beams, beams)
    length = torch.tensor([37, 11, 30], dtype=torch.int32)
    into = states if place else [_state(s, dtype, 50 + i) for i, s in enumerate(shapes)]
    want = [_want(x, parent, length, 2, y) for x, y in zip(states, into)]
    x = [t.to(dev) for t in states]
    got = B.beam_reorder(x, parent.to(dev), length.to(dev), out=None if place else [t.to(dev) for t in into])
    assert not got["status"].any()
    for g, w, a, b in zip(got["states"], want, x, states):
        assert torch.equal(g.cpu(), w)
        assert place or torch.equal(a.cpu(), b)


@pytest.mark.parametrize("place", [True, False])
def test_reorder_layouts(place):
    """Positions before the beams, heads before positions, keys and values in one tensor, padding between rows, states
    without positions, lengths of nothing and of one."""
    R, Bm = 4, 5
    parent, length = _parents(R, Bm, 3), torch.tensor([0, 1, 19, 20], dtype=torch.int32)

    def make(seed):
        t = _state((20, R, Bm, 8), torch.bfloat16, seed)                # positions outermost
        heads = _state((R, Bm, 3, 20, 16), torch.bfloat16, seed + 1)    # [.., heads, positions, ..]
        pair = _state((R, Bm, 20, 2, 64), torch.bfloat16, seed + 2)     # keys and values
        wide_ = _state((R, Bm, 24, 40), torch.bfloat16, seed + 3)       # rows of 30 inside rows of 40
        return t, heads, pair, wide_, _state((R, Bm), torch.float32, seed + 4), _state((R, Bm, 20, 7), torch.int8, seed + 5)

    def views(t, heads, pair, wide_, flat, odd):
        return [(t.permute(1, 2, 0, 3), 2), (heads, 3), (pair[:, :, :, 0], 2), (pair[:, :, :, 1], 2), (wide_[:, :, 1:21, 3:33], 2),
                (flat, 2), (odd, 2)]

    src, dst = make(1), make(1 if place else 100)
    on, to = [t.to(dev) for t in src], [t.to(dev) for t in dst]
    if place:
        to = on
    for axis in (2, 3):
        for (x, at), (y, _), (a, _), (b, _) in zip(views(*on), views(*to), views(*src), views(*dst)):
            if at == axis:
                b.copy_(_want(a, parent, length, axis, b))
        picked = [(x, y) for (x, at), (y, _) in zip(views(*on), views(*to)) if at == axis]
        got = B.beam_reorder([x for x, _ in picked], parent.to(dev), length.to(dev), axis=axis, out=None if place else [y for _, y in picked])
        assert not got["status"].any()
    for g, w in zip(to, dst):
        assert torch.equal(g.cpu(), w)  # what lies between the parts too


def test_reorder_many_states():
    R, Bm = 2, 4
    parent = _parents(R, Bm, 1)
    states = [_state((R, Bm, 10, 4 + 4 * (i % 3)), torch.float32, i) for i in range(35)]
    want = [_want(x, parent, None, 2, x) for x in states]
    got = B.beam_reorder([x.to(dev) for x in states], parent.to(dev))
    assert all(torch.equal(g.cpu(), w) for g, w in zip(got["states"], want))


def test_reorder_refused_requests():
    R, Bm = 5, 3
    x = _state((R, Bm, 12, 8), torch.float32, 1)
    parent = torch.tensor([[1, 2, 0]] * R, dtype=torch.int32)
    parent[1, 2], parent[2, 0] = 3, -2
    length = torch.tensor([12, 12, 12, 13, -1], dtype=torch.int32)
    got = B.beam_reorder([x.to(dev)], parent.to(dev), length.to(dev))
    assert got["status"].tolist() == [0, 24, 24, 25, 25]
    want = x.clone()
    want[0] = x[0, [1, 2, 0]]
    assert torch.equal(got["states"][0].cpu(), want)


def test_reorder_beyond_32_bits():
    """A state of more than 8 GiB."""
    R, Bm, T, D = 3, 3, 1 << 17, 4096
    x = torch.zeros((R, Bm, T, D), dtype=torch.bfloat16, device=dev)
    at = torch.arange(0, T, 9973, device=dev)
    x[:, :, at] = torch.arange(R * Bm, device=dev, dtype=torch.bfloat16).view(R, Bm, 1, 1) + 1
    x[:, :, T - 1, D - 1] = 40
    parent = torch.tensor([[2, 0, 1], [0, 0, 0], [1, 1, 2]], dtype=torch.int32, device=dev)
    length = torch.tensor([T, T, T - 1], dtype=torch.int32, device=dev)
    assert not B.beam_reorder([x], parent, length)["status"].any()
    for r in range(R):
        for b in range(Bm):
            assert (x[r, b, at] == r * Bm + int(parent[r, b]) + 1).all()
    assert (x[:, :, T - 1, D - 1] == 40).all() and not x[:, :, 1].any()


def test_reorder_on_streams_and_in_graphs():
    R, Bm = 4, 6
    x = [_state((R, Bm, 50, 32), torch.bfloat16, k).to(dev) for k in (1, 2)]
    parents = [_parents(R, Bm, k).clamp(min=0).to(dev) for k in (1, 2)]
    row = torch.arange(R, device=dev)[:, None]
    want = [[t[row, p.long()] for p in parents] for t in x]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in x]
    with torch.cuda.stream(s):
        B.beam_reorder([x[1]], parents[0], out=[out[1]])
    B.beam_reorder([x[0]], parents[0], out=[out[0]])
    torch.cuda.synchronize()
    assert all(torch.equal(out[i], want[i][0]) for i in (0, 1))
    p, t = parents[0].clone(), x[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.beam_reorder([t], p)
    for k in (1, 0, 1):
        t.copy_(x[k])
        p.copy_(parents[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t, want[k][k])


def test_reorder_refusals():
    p = torch.zeros((2, 3), dtype=torch.int32, device=dev)
    x = torch.zeros((2, 3, 8, 4), device=dev)
    with pytest.raises(ValueError):
        B.beam_reorder([], p)
    with pytest.raises(ValueError):
        B.beam_reorder([x[:1]], p)
    with pytest.raises(ValueError):
        B.beam_reorder([x], p.long())
    with pytest.raises(ValueError):
        B.beam_reorder([x[..., ::2]], p)
    with pytest.raises(ValueError):
        B.beam_reorder([x], p, out=[x[:, :, :4]])
    with pytest.raises(ValueError):
        B.beam_reorder([x], p, axis=1)
    for bad in (dict(states=[x, x]), dict(states=[torch.zeros((2, 1, 8, 4), device=dev).expand(2, 3, 8, 4)]),
                dict(states=[x, x.clone()], out=[x, torch.empty_like(x)])):
        with pytest.raises(B.DsparkError):
            B.beam_reorder(parent=p, **bad)
    y = torch.zeros((2, 6, 8, 4), device=dev)
    with pytest.raises(B.DsparkError):
        B.beam_reorder([y[:, :3]], p, out=[y[:, 1:4]])


def test_reorder_counts_as_written():
    """A backward pass that saved a state refuses it once it has been reordered."""
    x = torch.zeros((2, 3, 8, 4), device=dev)
    w = torch.ones(4, device=dev, requires_grad=True)
    y = (x * w).sum()
    B.beam_reorder([x], torch.zeros((2, 3), dtype=torch.int32, device=dev))
    with pytest.raises(RuntimeError):
        y.backward()
