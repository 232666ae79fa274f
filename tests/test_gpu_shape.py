"""Shaping of logits against the 64-bit definition.

Tolerance, counted before the first run: a shaped logit is built from at most
the quotient or product with the repetition penalty, the product with the
frequency, two subtractions and the sum with the bias (each off by half a
binary32 step, 2^-24, of at most the sum of the magnitudes), the reciprocal of
the temperature and the product with it (2^-24 of the value each): 7 x 2^-24
of the magnitudes; a bf16 result adds 2^-8 of the value."""
import numpy as np
import pytest
import torch

from oracle import logits as L
from vocab_wide_draft_amd import binding as B
from vocab_wide_draft_amd import workloads as W

from gpu_helpers import dev, to_dev

pytestmark = pytest.mark.gpu
F = 2.0 ** -24


def rows_of(rng, n, V, dtype, scale=3.0):
    x = (rng.standard_normal((n, V)) * scale).astype(np.float32)
    return W.f32_to_bf16_bits(x) if dtype == "bf16" else x


def f64(a, dtype):
    return (W.bf16_bits_to_f32(a) if dtype == "bf16" else a).astype(np.float64)


def host64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(got, want, mag, out_bf16, label=""):
    got = np.asarray(got, np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), label
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), label
    assert np.isfinite(got[fin]).all(), label
    tol = 7.001 * F * mag[fin] * (1 + 2.0 ** -8) + (2.0 ** -8 * np.abs(want[fin]) if out_bf16 else 0.0) + 2.0 ** -133
    bad = np.abs(got[fin] - want[fin]) > tol
    assert not bad.any(), (label, got[fin][bad][:4], want[fin][bad][:4])


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dev())


def pack(allowed, extra=0):
    """bool [m, V] -> int32 words, with `extra` unused words a row; bits past V are set."""
    m, V = allowed.shape
    w = (V + 31) // 32
    bits = np.ones((m, w * 32), np.uint8)
    bits[:, :V] = allowed
    words = np.packbits(bits.reshape(m, w, 4, 8), axis=3, bitorder="little").reshape(m, w * 4).view(np.int32)
    out = np.full((m, w + extra), 0x5A5A5A5A, np.int32)
    out[:, :w] = words
    return out


def case(rng, R, P, V, H, nb, masked):
    """Everything at once, ragged."""
    c = {"hist": rng.integers(0, V, (R, H)), "len": rng.integers(0, H + 1, R)}
    c["len"][0] = H
    if H:
        c["hist"][:, : H // 2] = rng.integers(0, min(V, 5), (R, H // 2))  # repeated ids
    if R > 1:
        c["len"][1] = 0
    if R > 2 and H:
        c["len"][2] = 1
    c["plen"] = np.array([rng.integers(0, n + 1) for n in c["len"]])
    c["draft"] = rng.integers(0, V, (R, max(P - 1, 1)))
    if P > 2:
        c["draft"][:, 1] = c["draft"][:, 0]  # the same id twice
    c["rep"] = rng.uniform(0.6, 1.8, R).astype(np.float32)
    c["freq"] = rng.uniform(-0.5, 1.0, R).astype(np.float32)
    c["pres"] = rng.uniform(-0.5, 1.0, R).astype(np.float32)
    c["temp"] = rng.uniform(0.3, 2.0, R).astype(np.float32)
    c["bias"] = []
    for r in range(R):
        n = 0 if r % 3 == 1 else min(nb, V)
        ids = np.sort(rng.permutation(V)[:n])
        val = rng.normal(0, 3, n).astype(np.float32)
        val[::7] = -np.inf
        c["bias"].append(list(zip(ids.tolist(), val.tolist())))
    if masked:
        c["allowed"] = rng.random((3, V)) < np.array([[0.05], [0.9], [0.0]])
        c["mask_row"] = rng.integers(-1, 3, R * P)
        c["mask_row"][0] = 2  # nothing allowed
    return c


def call(c, x, P, **kw):
    off = np.cumsum([0] + [len(b) for b in c["bias"]])
    flat = [e for b in c["bias"] for e in b]
    bias = (torch.from_numpy(off.astype(np.int64)).to(dev()), i32([e[0] for e in flat]), f32([e[1] for e in flat]))
    if "allowed" in c:
        kw.update(mask=i32(pack(c["allowed"], extra=3))[:, : (x.shape[1] + 31) // 32 + 1], mask_row=i32(c["mask_row"]))
    return B.shape_logits(x, P, history=i32(c["hist"]), history_len=i32(c["len"]), prompt_len=i32(c["plen"]),
                          draft=i32(c["draft"]), repetition=f32(c["rep"]), frequency=f32(c["freq"]),
                          presence=f32(c["pres"]), temperature=f32(c["temp"]), bias=bias, **kw)


def want(c, x, P, j):
    r, i = divmod(j, P)
    n, pl = int(c["len"][r]), int(c["plen"][r])
    made = c["hist"][r, pl:n].tolist() + c["draft"][r, :i].tolist()
    m = int(c["mask_row"][j]) if "allowed" in c else -1
    return L.shape_row(x[j], c["hist"][r, :pl].tolist(), made, float(c["rep"][r]), float(c["freq"][r]),
                       float(c["pres"][r]), float(c["temp"][r]), c["bias"][r], c["allowed"][m] if m >= 0 else None)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("R,P,V,H,nb", [(1, 1, 1, 0, 1), (1, 6, 7, 3, 2), (3, 1, 8, 9, 8), (4, 5, 31, 40, 3),
                                        (3, 6, 33, 1, 33), (5, 2, 2047, 100, 40), (2, 6, 2049, 300, 700),
                                        (3, 3, 20003, 1000, 100)])
def test_shape_everything(dtype, out, R, P, V, H, nb):
    rng = np.random.default_rng(R * 1000 + V)
    a = rows_of(rng, R * P, V, dtype)
    c = case(rng, R, P, V, H, nb, True)
    x = to_dev(a, dtype)
    before = x.clone()
    g = call(c, x, P, out_dtype=torch.float32 if out == "f32" else None)
    torch.cuda.synchronize()
    assert (g["status"] == 0).all() and torch.equal(x.view(torch.int16 if dtype == "bf16" else torch.int32), before.view(torch.int16 if dtype == "bf16" else torch.int32))
    got = host64(g["logits"])
    for j in range(R * P):
        w, mag = want(c, f64(a, dtype), P, j)
        check(got[j], w, mag, out == "bf16", (j,))


@pytest.mark.parametrize("V,R,P", [(129280, 2, 6), (131080, 1, 1), (129280, 70, 1)])
def test_shape_long_rows(V, R, P):
    rng = np.random.default_rng(V + R)
    a = rows_of(rng, R * P, V, "bf16")
    c = case(rng, R, P, V, 3000, 200, R < 10)
    g = call(c, to_dev(a, "bf16"), P, out_dtype=torch.float32)
    got = host64(g["logits"])
    for j in list(range(min(R * P, 12))) + [R * P - 1]:
        w, mag = want(c, {j: f64(a[j], "bf16")}, P, j)
        check(got[j], w, mag, False, (j,))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shape_in_place_and_padding_untouched(dtype):
    rng = np.random.default_rng(7)
    R, P, V = 3, 5, 1001
    a = rows_of(rng, R * P, V, dtype)
    c = case(rng, R, P, V, 60, 9, True)
    apart = call(c, to_dev(a, dtype), P)
    wide = to_dev(np.concatenate([a, rows_of(rng, R * P, 31, dtype)], 1), dtype)  # 31 values behind each row
    x = wide[:, :V]
    tail = wide[:, V:].clone()
    g = call(c, x, P, out=x)
    assert g["logits"].data_ptr() == x.data_ptr()
    assert torch.equal(x.float(), apart["logits"].float())
    assert torch.equal(wide[:, V:].float(), tail.float())
    o = torch.full((R * P, 1024), 7.0, dtype=x.dtype, device=dev())
    call(c, to_dev(a, dtype), P, out=o[:, :V])
    assert torch.equal(o[:, :V].float(), apart["logits"].float()) and (o[:, V:] == 7.0).all()


def test_shape_steps_one_by_one():
    """Each step alone; the others left out (None) or neutral."""
    rng = np.random.default_rng(11)
    V, R = 300, 2
    a = rows_of(rng, R, V, "f32")
    x = to_dev(a, "f32")
    same = B.shape_logits(x)["logits"]
    assert torch.equal(same, x)
    hist = rng.integers(0, V, (R, 50))
    only = {"repetition": dict(rep=1.3), "frequency": dict(freq=0.4), "presence": dict(pres=-0.3)}
    for name, kw in only.items():
        v = f32([list(kw.values())[0]] * R)
        g = host64(B.shape_logits(x, history=i32(hist), **{name: v})["logits"])
        for r in range(R):
            w, mag = L.shape_row(a[r], (), hist[r], **{k: float(np.float32(t)) for k, t in kw.items()})
            check(g[r], w, mag, False, name)
    # a prompt's tokens feel the repetition penalty alone
    g = host64(B.shape_logits(x, history=i32(hist), prompt_len=i32([50, 50]), repetition=f32([1.5, 1.5]),
                              frequency=f32([1.0, 1.0]), presence=f32([1.0, 1.0]))["logits"])
    for r in range(R):
        w, mag = L.shape_row(a[r], hist[r], (), rep=1.5, freq=1.0, pres=1.0)
        check(g[r], w, mag, False)
    # neutral penalties: history and draft are not read, so nothing in them is refused
    g = B.shape_logits(x, history=i32(np.full((R, 4), -9)), history_len=i32([99, -1]), repetition=f32([1, 1]))
    assert (g["status"] == 0).all() and torch.equal(g["logits"], x)
    # drafted tokens count without a history
    a6 = rows_of(rng, 6, V, "f32")
    g = host64(B.shape_logits(to_dev(a6, "f32"), 6, draft=i32([[5, 5, 9, 5, 1]]), frequency=f32([0.5]))["logits"])
    for i in range(6):
        w, mag = L.shape_row(a6[i], (), [5, 5, 9, 5, 1][:i], freq=0.5)
        check(g[i], w, mag, False, i)


def test_shape_masks_and_special_values():
    V = 70
    low = np.float32(-3.3895314e38)  # the lowest finite bf16
    a = np.zeros((6, V), np.float32)
    a[0, ::2] = np.nan
    a[1, ::2] = np.inf
    a[2, :] = -np.inf
    a[3, :] = low
    a[4, :] = np.float32(3.0e38)
    a[5, 1:] = np.nan
    allowed = np.zeros((2, V), bool)
    allowed[0, 1::2] = True
    words = i32(pack(allowed))
    for dtype in ("f32", "bf16"):
        x = to_dev(W.f32_to_bf16_bits(np.nan_to_num(a, nan=9.0, posinf=np.inf, neginf=-np.inf)) if dtype == "bf16" else a, dtype)
        g = B.shape_logits(x, mask=words, mask_row=i32([0, 0, 0, 0, 1, 1]))
        y = host64(g["logits"])
        assert (g["status"] == 0).all()
        assert (y[:, ::2] == -np.inf).all()  # NaN and +inf under the mask are gone
        assert (y[0, 1::2] == 0).all() and (y[1, 1::2] == 0).all() and (y[2] == -np.inf).all()
        assert (y[3, 1::2] == float(low) if dtype == "f32" else np.abs(y[3, 1::2] / low - 1) < 2.0 ** -8).all()
        assert (y[4:] == -np.inf).all()  # a mask that allows nothing
    # unmasked: the arithmetic applies; -inf stays -inf under a penalty, NaN stays NaN
    x = to_dev(a, "f32")
    g = host64(B.shape_logits(x, history=i32(np.arange(70)[None].repeat(6, 0)), repetition=f32([2.0] * 6),
                              presence=f32([1.0] * 6), temperature=f32([0.5] * 6))["logits"])
    assert np.isnan(g[0, ::2]).all() and (g[1, ::2] == np.inf).all() and (g[2] == -np.inf).all()
    assert (g[3] == -np.inf).all()  # lowest value times two overflows


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("R,P,H", [(3, 1, 20000), (3, 6, 20000), (60, 2, 17000), (70, 1, 100), (70, 3, 100)])
def test_shape_every_kernel_choice(dtype, out, R, P, H):
    """Few and many requests, short and long histories, few and many rows each (V above one workgroup's slice)."""
    rng = np.random.default_rng(R + P)
    V = 70003
    a = rows_of(rng, R * P, V, dtype)
    c = case(rng, R, P, V, H, 30, True)
    g = call(c, to_dev(a, dtype), P, out_dtype=torch.float32 if out == "f32" else None)
    assert (g["status"] == 0).all()
    got = g["logits"]
    for j in sorted({0, P - 1, P, 2 * P - 1, R * P - 1}):
        w, mag = want(c, {j: f64(a[j], dtype)}, P, j)
        check(host64(got[j]), w, mag, out == "bf16", j)


def test_shape_counts_beyond_16_bits_and_long_history():
    rng = np.random.default_rng(3)
    V, H = 5000, 200_000
    a = rows_of(rng, 1, V, "f32")
    hist = np.full((1, H), 17)
    hist[0, ::2] = rng.integers(0, V, H // 2)
    g = host64(B.shape_logits(to_dev(a, "f32"), history=i32(hist), prompt_len=i32([10]), frequency=f32([0.001]),
                              repetition=f32([1.1]))["logits"])
    w, mag = L.shape_row(a[0], hist[0, :10], hist[0, 10:], rep=float(np.float32(1.1)), freq=float(np.float32(0.001)))
    check(g[0], w, mag, False)


def test_shape_refused_rows():
    rng = np.random.default_rng(9)
    V, P = 3001, 6
    R = 12
    a = rows_of(rng, R * P, V, "f32")
    c = case(rng, R, P, V, 20, 12, True)
    c["len"][:] = 20
    c["plen"][:] = 4
    c["bias"] = [[(3, 1.0), (9, 2.0), (2500, -1.0)] for _ in range(R)]
    exp = np.zeros((R, P), int)
    c["hist"][1, 19] = V; exp[1] = L.ST_BAD_HISTORY
    c["hist"][2, 0] = -1; exp[2] = L.ST_BAD_HISTORY
    c["len"][3] = 21; exp[3] = L.ST_BAD_HISTORY
    c["plen"][4] = 21; exp[4] = L.ST_BAD_HISTORY
    c["draft"][5, 2] = V; exp[5, 3:] = L.ST_BAD_HISTORY
    c["rep"][6] = 0.0; exp[6] = L.ST_BAD_PENALTY
    c["temp"][7] = np.inf; exp[7] = L.ST_BAD_PENALTY
    c["pres"][8] = np.nan; exp[8] = L.ST_BAD_PENALTY
    c["bias"][9] = [(3, 1.0), (3, 2.0), (2500, -1.0)]; exp[9] = L.ST_BAD_BIAS
    c["bias"][10] = [(3, 1.0), (9, float("nan")), (V, -1.0)]; exp[10] = L.ST_BAD_BIAS
    c["bias"][11] = [(-1, 1.0), (9, 2.0), (2500, float("inf"))]; exp[11] = L.ST_BAD_BIAS
    c["temp"][11] = -1.0; exp[11] = L.ST_BAD_PENALTY  # the smallest code
    c["mask_row"][0] = 3; exp[0, 0] = L.ST_BAD_MASK
    c["mask_row"][1] = -2; exp[0, 1] = L.ST_BAD_MASK
    g = call(c, to_dev(a, "f32"), P)
    st = g["status"].cpu().numpy().reshape(R, P)
    assert (st == exp).all(), (st, exp)
    got = host64(g["logits"])
    for j in range(R * P):
        if exp.flat[j]:
            assert (got[j] == -np.inf).all()
        else:
            w, mag = want(c, a, P, j)
            check(got[j], w, mag, False, j)
    # bias offsets that leave the lists or run backwards
    off = torch.tensor([0, 2, 1, 4, 3], device=dev())
    g = B.shape_logits(to_dev(a[:4], "f32"), bias=(off, i32([1, 2, 5]), f32([1, 1, 1])))
    assert g["status"].tolist() == [0, L.ST_BAD_BIAS, L.ST_BAD_BIAS, L.ST_BAD_BIAS]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shape_many_rows_of_one_request(dtype):
    """More rows than a wave has lanes, each with a mask and a drafted token of its own."""
    rng = np.random.default_rng(44)
    R, P, V = 2, 150, 2500
    a = rows_of(rng, R * P, V, dtype)
    c = case(rng, R, P, V, 30, 10, False)
    c["allowed"] = rng.random((40, V)) < 0.7
    c["mask_row"] = rng.integers(-1, 40, R * P)
    c["draft"][1, 100] = V  # the rows after it are refused
    g = call(c, to_dev(a, dtype), P)
    st = g["status"].cpu().numpy().reshape(R, P)
    assert not st[0].any() and not st[1, :101].any() and (st[1, 101:] == L.ST_BAD_HISTORY).all()
    got = host64(g["logits"])
    for j in range(R * P):
        if st.flat[j]:
            assert (got[j] == -np.inf).all()
        else:
            w, mag = want(c, f64(a, dtype), P, j)
            check(got[j], w, mag, dtype == "bf16", j)


def test_shape_factor_ranges():
    x = torch.ones((6, 64), device=dev())
    lo, hi = 2.0 ** -100, 2.0 ** 100
    hist = i32(np.zeros((6, 1)))
    r = f32([lo, hi, 2.0 ** -101, 2.0 ** 101, np.inf, -1.0])
    g = B.shape_logits(x, history=hist, repetition=r)
    assert g["status"].tolist() == [0, 0] + [L.ST_BAD_PENALTY] * 4
    assert g["logits"][:2, 0].tolist() == [hi, lo] and (g["logits"][:2, 1:] == 1).all()
    g = B.shape_logits(x, temperature=r)
    assert g["status"].tolist() == [0, 0] + [L.ST_BAD_PENALTY] * 4
    assert (g["logits"][0] == hi).all() and (g["logits"][1] == lo).all() and (g["logits"][2:] == -np.inf).all()


def test_shape_mask_per_row_without_index():
    rng = np.random.default_rng(2)
    a = rows_of(rng, 4, 129, "bf16")
    allowed = rng.random((4, 129)) < 0.5
    g = host64(B.shape_logits(to_dev(a, "bf16"), mask=i32(pack(allowed)))["logits"])
    assert np.array_equal(g, np.where(allowed, f64(a, "bf16"), -np.inf))


def test_shape_far_rows():
    """Rows whose offset passes 2^31 elements."""
    n, V = 16700, 129280
    x = torch.zeros((n, V), dtype=torch.bfloat16, device=dev())
    x[-1] = 2.0
    hist = torch.zeros((n, 1), dtype=torch.int32, device=dev())
    g = B.shape_logits(x, history=hist, frequency=torch.ones(n, device=dev()), out=x)
    assert (g["status"] == 0).all()
    assert x[-1, 0] == 1.0 and (x[-1, 1:] == 2.0).all() and x[0, 0] == -1.0 and (x[1, 1:] == 0).all()


def test_shape_other_stream_and_graph_replays():
    rng = np.random.default_rng(21)
    R, P, V = 4, 6, 5003
    a = rows_of(rng, R * P, V, "bf16")
    c = case(rng, R, P, V, 200, 20, True)
    x = to_dev(a, "bf16")
    ref = call(c, x, P)["logits"].float()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = call(c, x, P)["logits"].float()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, ref)
    args = dict(history=i32(c["hist"]), history_len=i32(c["len"]), prompt_len=i32(c["plen"]), draft=i32(c["draft"]),
                repetition=f32(c["rep"]), frequency=f32(c["freq"]), presence=f32(c["pres"]), temperature=f32(c["temp"]))
    eager = B.shape_logits(x, P, **args)["logits"].clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.shape_logits(x, P, **args))
        graphs.append(g)
    for rep in range(3):
        for g, o in zip(graphs, outs):
            o["logits"].zero_()
            g.replay()
        again = B.shape_logits(x, P, **args)["logits"]
        torch.cuda.synchronize()
        for o in outs + [{"logits": again}]:
            assert torch.equal(o["logits"].view(torch.int16), eager.view(torch.int16)), rep


def test_shape_arguments_inside_wider_buffers():
    rng = np.random.default_rng(46)
    R, P, V = 3, 6, 5000
    a = rows_of(rng, R * P, V, "bf16")
    c = case(rng, R, P, V, 70, 12, False)
    want_ = call(c, to_dev(a, "bf16"), P)["logits"]
    wide_h, wide_d = i32(np.full((R, 90), -7)), i32(np.full((R, 11), V + 5))
    wide_h[:, 8:78] = i32(c["hist"])
    wide_d[:, 3:8] = i32(c["draft"])
    off = np.cumsum([0] + [len(b) for b in c["bias"]])
    flat = [e for b in c["bias"] for e in b]
    g = B.shape_logits(to_dev(a, "bf16"), P, history=wide_h[:, 8:78], history_len=i32(c["len"]), prompt_len=i32(c["plen"]),
                       draft=wide_d[:, 3:8], repetition=f32(c["rep"]), frequency=f32(c["freq"]), presence=f32(c["pres"]),
                       temperature=f32(c["temp"]),
                       bias=(torch.from_numpy(off.astype(np.int64)).to(dev()), i32([e[0] for e in flat]), f32([e[1] for e in flat])))
    assert not g["status"].any() and torch.equal(g["logits"].view(torch.int16), want_.view(torch.int16))


def test_shape_a_bias_for_every_token():
    rng = np.random.default_rng(47)
    V = 30001
    a = rows_of(rng, 2, V, "f32")
    val = rng.normal(0, 1, 2 * V).astype(np.float32)
    off = torch.tensor([0, V, 2 * V], device=dev())
    g = host64(B.shape_logits(to_dev(a, "f32"), bias=(off, i32(np.tile(np.arange(V), 2)), f32(val)))["logits"])
    w = a.astype(np.float64) + val.reshape(2, V)
    assert (np.abs(g - w) <= F * np.abs(w) + 2.0 ** -133).all()


def test_shape_empty_arguments():
    x = torch.ones((3, 40), device=dev())
    two = f32([2.0] * 3)
    empty = torch.zeros((3, 0), dtype=torch.int32, device=dev())
    g = B.shape_logits(x, history=empty, history_len=i32([0, 1, 0]), presence=two)
    assert g["status"].tolist() == [0, L.ST_BAD_HISTORY, 0] and (g["logits"][0] == 1).all()
    g = B.shape_logits(x, history=empty, presence=two)
    assert not g["status"].any() and torch.equal(g["logits"], x)
    off = torch.zeros(4, dtype=torch.int64, device=dev())
    g = B.shape_logits(x, bias=(off, i32([]), f32([])))
    assert not g["status"].any() and torch.equal(g["logits"], x)
    with pytest.raises(ValueError):
        B.shape_logits(x, mask=torch.zeros((0, 2), dtype=torch.int32, device=dev()), mask_row=i32([0, 0, 0]))


@pytest.mark.parametrize("how", ["bias without offsets", "bias without values", "masks' rows without masks",
                                 "lengths without a history", "prompts without a history"])
def test_shape_incomplete_arguments(how):
    """An argument that its missing partner would leave without effect is refused."""
    x = torch.ones((3, 40), device=dev())
    off, three = torch.tensor([0, 1, 1, 1], device=dev()), i32([1, 1, 1])
    kw = {"bias without offsets": {"bias": (None, i32([4]), f32([1.0]))},
          "bias without values": {"bias": (off, i32([4]), None)},
          "masks' rows without masks": {"mask_row": three},
          "lengths without a history": {"history_len": three},
          "prompts without a history": {"prompt_len": three}}[how]
    with pytest.raises(ValueError):
        B.shape_logits(x, **kw)


def test_shape_no_rows():
    g = B.shape_logits(torch.zeros((0, 64), device=dev()), 6)
    assert g["logits"].shape == (0, 64) and g["status"].shape == (0,)
