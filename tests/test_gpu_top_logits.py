"""Top logits and the row's log-sum-exp against the 64-bit definition: ids,
logits and lengths equal; lse within a bound counted before the first run:
an exponent (x - m) c has three roundings of 2^-24 of itself (difference,
product, c), the hardware exponential is off by 2^-23, a thread adds at most
160 binary32 values before binary64 takes over (2^-24 each), and the result
is rounded once."""
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


def lse_tol(x, temp):
    """Bound of |lse - exact| for a row (float64) without NaN."""
    u = x[x > -np.inf] / temp
    w = np.exp(u - u.max())
    t = np.abs(u - u.max())  # natural units: 2^-24 of t each, as exp2 takes t log2 e
    return F * ((w * (3 * t + 2)).sum() / w.sum() + 160) + F * abs(L.logsumexp(u))


def check_rows(a, dtype, ks, temp, g, rows=None):
    ids, z, ln, lse, st = (g[k].cpu().numpy() for k in ("ids", "logits", "len", "lse", "status"))
    for r in range(a.shape[0]) if rows is None else rows:
        x = f64(a[r], dtype)
        s, wi, wz, wl = L.top_row(x, int(ks[r]), temp)
        assert st[r] == s, (r, st[r], s)
        n = len(wi)
        assert ln[r] == n, (r, ln[r], n)
        assert (ids[r, :n] == wi).all() and not ids[r, n:].any(), r
        assert (z[r, :n].astype(np.float64) == wz).all() and not z[r, n:].any(), r
        if s == L.ST_OK:
            assert abs(float(lse[r]) - wl) <= lse_tol(x, temp), (r, lse[r], wl)
        else:
            assert lse[r] == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(1, 1), (2, 5), (7, 3), (8, 8), (33, 1), (1000, 1000), (1025, 1024), (4097, 100),
                                 (20003, 1), (20003, 1024), (70001, 257)])
def test_top_small(dtype, V, k):
    rng = np.random.default_rng(V * 7 + k)
    a = rows_of(rng, 5, V, dtype)
    g = B.top_logits(to_dev(a, dtype), k, temperature=0.7)
    check_rows(a, dtype, [k] * 5, 0.7, g)


@pytest.mark.parametrize("dtype,V", [("bf16", 129280), ("bf16", 131072), ("bf16", 131073), ("f32", 129280),
                                     ("f32", 200001)])
@pytest.mark.parametrize("n", [1, 6])
def test_top_long(dtype, V, n):
    rng = np.random.default_rng(V + n)
    a = rows_of(rng, n, V, dtype)
    ks = np.array([1024, 1, 0, 50, 333, 1023][:n], np.int32)
    g = B.top_logits(to_dev(a, dtype), 1024, topk=torch.from_numpy(ks).to(dev()), temperature=2.0)
    check_rows(a, dtype, ks, 2.0, g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2048, 2049, 4096, 8192, 8193, 16384, 16385, 16391, 24577])
@pytest.mark.parametrize("k", [7, 1024])
def test_top_around_the_sizes_where_the_kernel_changes(dtype, V, k):
    rng = np.random.default_rng(V + k)
    a = rows_of(rng, 3, V, dtype)
    g = B.top_logits(to_dev(a, dtype), k, temperature=1.3)
    check_rows(a, dtype, [k] * 3, 1.3, g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(4096, 30), (4097, 30), (8000, 200), (8000, 900), (16384, 1024)])
def test_top_many_rows_of_middle_length(dtype, V, k):
    rng = np.random.default_rng(V + 3 * k)
    a = np.tile(rows_of(rng, 20, V, dtype), (27, 1))
    a[7] = special_rows(rng, V, dtype)[6]  # ties
    g = B.top_logits(to_dev(a, dtype), k)
    check_rows(a, dtype, [k] * 540, 1.0, g, rows=list(range(20)) + [539])
    for name in g:
        assert torch.equal(g[name][20:].view(26, 20, -1), g[name][20:40].view(1, 20, -1).expand(26, 20, -1)), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_top_where_the_sample_misleads(dtype):
    """The largest logits all inside, or all outside, the sampled runs."""
    rng = np.random.default_rng(77)
    V, k = 40003, 600
    step = (V // 64) & ~7
    sampled = np.zeros(V, bool)
    for c in range(64):
        sampled[c * step:c * step + 32] = True
    x = (rng.standard_normal((4, V)) * 2).astype(np.float32)
    x[0, sampled] += 40.0                       # a threshold above nearly all of the top k
    x[1, ~sampled] += 40.0                      # one below nearly all logits
    x[2, 100:100 + k] += 60.0                   # the top k in one slice
    x[3, ::2] = -np.inf
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    g = B.top_logits(to_dev(a, dtype), k)
    check_rows(a, dtype, [k] * 4, 1.0, g)


def special_rows(rng, V, dtype):
    x = (rng.standard_normal((14, V)) * 2).astype(np.float32)
    x[0, rng.random(V) < 0.5] = -np.inf
    x[1, :] = -np.inf
    x[1, [3, V - 1]] = [1.0, -2.0]              # fewer finite logits than k
    x[2, :] = -np.inf                           # none
    x[3, V // 2] = np.nan
    x[4, V - 1] = np.inf
    x[5, :] = 1.5                               # one value
    x[6] = rng.integers(0, 3, V) - 1.0          # ties, +0 among them
    x[7] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    x[8] = -np.abs(x[8]) - 1.0                  # all negative
    x[9, :] = np.float32(-3.3895314e38)         # the lowest finite bf16
    x[9, 5] = np.float32(3.3895314e38)
    x[10, :] = np.float32(1e-39)                # subnormal
    x[11] = np.sort(x[11])                      # the largest at the end
    x[12] = np.sort(x[12])[::-1]
    x[13, :] = -30.0
    x[13, 7] = 60.0                             # all mass on one
    return W.f32_to_bf16_bits(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf)) if dtype == "bf16" else x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(257, 40), (5000, 1024), (129280, 64)])
def test_top_special(dtype, V, k):
    rng = np.random.default_rng(V)
    a = special_rows(rng, V, dtype)
    if dtype == "bf16":
        a[3, V // 2] = 0xFFC1  # a negative NaN
    g = B.top_logits(to_dev(a, dtype), k)
    check_rows(a, dtype, [k] * 14, 1.0, g)
    # more rows than workgroups that fit at once: the same answers
    many = np.tile(a, (40, 1))
    h = B.top_logits(to_dev(many, dtype), k)
    for name in ("ids", "logits", "len", "lse", "status"):
        assert torch.equal(h[name].view(40, 14, -1), g[name].view(1, 14, -1).expand(40, 14, -1)), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 20003])
@pytest.mark.parametrize("temp", [2.0 ** -100, 2.0 ** -10, 2.0 ** 10, 2.0 ** 100])
def test_top_extreme_temperatures(dtype, V, temp):
    rng = np.random.default_rng(V)
    a = rows_of(rng, 4, V, dtype)
    check_rows(a, dtype, [20] * 4, temp, B.top_logits(to_dev(a, dtype), 20, temperature=temp))


def test_top_refused_k_and_k0():
    rng = np.random.default_rng(4)
    for dtype in ("bf16", "f32"):
        a = rows_of(rng, 4, 100, dtype)
        g = B.top_logits(to_dev(a, dtype), 128, topk=torch.tensor([-1, 101, 100, 0], dtype=torch.int32, device=dev()))
        assert g["status"].tolist() == [L.ST_BAD_TOPK, L.ST_BAD_TOPK, 0, 0]
        assert g["len"].tolist() == [0, 0, 100, 0] and g["lse"][:2].tolist() == [0.0, 0.0] and not g["ids"][:2].any()
        h = B.top_logits(to_dev(a, dtype), 0)
        assert h["ids"].shape == (4, 0) and h["len"].tolist() == [0] * 4 and torch.equal(h["lse"][2:], g["lse"][2:])
        check_rows(a, dtype, [0, 0, 100, 0], 1.0, g, rows=[2, 3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_top_strides_stream_and_graph(dtype):
    rng = np.random.default_rng(8)
    V, n = 3003, 9
    a = rows_of(rng, n, V + 21, dtype)
    x = to_dev(a, dtype)[:, :V]  # values behind every row
    ref = B.top_logits(x, 100)
    check_rows(a[:, :V], dtype, [100] * n, 1.0, ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = B.top_logits(x, 100)
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.top_logits(x, 100))
        graphs.append(g)
    for rep in range(3):
        for g, o in zip(graphs, outs):
            for k in o:
                o[k].fill_(7)
            g.replay()
        e = B.top_logits(x, 100)
        torch.cuda.synchronize()
        for o in outs + [e, y]:
            for k in ref:
                assert torch.equal(o[k], ref[k]), (rep, k)


def test_top_far_rows():
    n, V = 16700, 129280
    x = torch.zeros((n, V), dtype=torch.bfloat16, device=dev())
    x[-1, 77] = 3.0
    g = B.top_logits(x, 2)
    assert g["ids"][-1].tolist() == [0, 77] and g["ids"][0].tolist() == [0, 1] and (g["len"] == 2).all()


def test_top_no_rows():
    g = B.top_logits(torch.zeros((0, 64), device=dev()), 4)
    assert g["ids"].shape == (0, 4)
