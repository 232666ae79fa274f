"""Distillation loss and gradient against the 64-bit definition, and the
gradient against differences of the loss.

Tolerances, counted before the first run (F = 2^-24): a sum of exponentials
is off by D = F (3 t + 2 + 160) relative, t the mean of |u - max u| under the
softmax, as for the log-sum-exp of top logits.  The list's side is binary64.
So the loss is off by D times the mass that multiplies it, 2 at most (log S
and log Q), and F of itself; q_v by D + F (3 t_v + 6); 1 - P / Q by D P / Q;
p_v by F (its rounding) and the products by 3 F each; bf16 adds 2^-8."""
import numpy as np
import pytest
import torch
import torch.utils.checkpoint

from oracle import logits as L
from vocab_wide_draft_amd import binding as B
from vocab_wide_draft_amd import workloads as W

from gpu_helpers import dev, to_dev
from test_gpu_shape import f32, f64, host64, i32, rows_of

pytestmark = pytest.mark.gpu
F = 2.0 ** -24


def lists(rng, x, k, temp, tail, ragged=True):
    """A teacher near the student rows x (float64)."""
    n, V = x.shape
    z = (np.where(np.isfinite(x), x, 0.0) * 0.7 + rng.normal(0, 1.0, (n, V))).astype(np.float32)
    ids, zl = np.zeros((n, k), np.int32), np.zeros((n, k), np.float32)
    ln = np.full(n, min(k, V))
    if ragged:
        ln = rng.integers(1, min(k, V) + 1, n)
        ln[0] = min(k, V)
        if n > 2:
            ln[2] = 0
    for r in range(n):
        top = np.sort(np.argsort(-z[r], kind="stable")[:ln[r]])
        ids[r, :ln[r]], zl[r, :ln[r]] = top, z[r, top]
        ids[r, ln[r]:], zl[r, ln[r]:] = -5, np.nan  # what lies behind a list is not read
    lse = np.array([L.logsumexp(z[r].astype(np.float64) / temp) for r in range(n)], np.float32)
    return ids, zl, ln.astype(np.int32), lse if tail else None


def teacher(t):
    return {"ids": i32(t[0]), "logits": f32(t[1]), "len": i32(t[2]), "lse": None if t[3] is None else f32(t[3])}


def check(a, dtype, t, temp, weight, loss, grad, rows=None):
    ids, zl, ln, lse = t
    for r in range(a.shape[0]) if rows is None else rows:
        x = f64(a[r], dtype)
        n = int(ln[r])
        if n == 0:
            assert loss[r] == 0 and (grad is None or (grad[r] == 0).all())
            continue
        wl, wg, q, p, P, Q = L.distill_row(x, ids[r, :n], zl[r, :n], temp, None if lse is None else lse[r])
        u = x / temp
        with np.errstate(invalid="ignore"):
            tv = np.where(x > -np.inf, u.max() - u, 0.0)
        D = F * (3 * (q * tv).sum() + 162)
        if np.isinf(wl):
            assert loss[r] == wl, r
        else:
            assert abs(loss[r] - wl) <= 2 * D * max(1.0, p.sum()) + F * abs(wl) + 1e-12, (r, loss[r], wl)
        if grad is not None:
            w = float(weight[r])
            ratio = P / Q if P > 0 else 0.0
            # the hardware exponential gives 0 for a result below the smallest normal 2^-126, which is off by less
            # than 2^-126 and is multiplied by at most (1 + P / Q) w / T (1 / S <= 1, as the largest term of S is 1)
            tol = np.abs(w / temp) * ((q * (D + F * (3 * tv + 6)) + 2.0 ** -126) * (1 + 2 * ratio) + 4 * F * (p + q)) + 2.0 ** -133
            want = wg * w
            if dtype == "bf16":
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
            bad = np.abs(grad[r] - want) > tol
            assert not bad.any(), (r, np.flatnonzero(bad)[:5], grad[r][bad][:5], want[bad][:5], tol[bad][:5])


def run_all(a, dtype, t, temp, weight, rows=None):
    x, tt, w = to_dev(a, dtype), teacher(t), f32(weight)
    f = B.distill(x, tt, temp)
    g = B.distill_backward(x, tt, f, w, temp)
    s = B.distill_step(x, tt, w, temp)
    torch.cuda.synchronize()
    assert (f["status"] == 0).all() and (s["status"] == 0).all()
    check(a, dtype, t, temp, weight, f["loss"].cpu().numpy(), host64(g), rows)
    check(a, dtype, t, temp, weight, s["loss"].cpu().numpy(), host64(s["grad"]), rows)
    return x, tt, w, f, g, s


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k,n", [(1, 1, 1), (2, 1, 3), (7, 3, 3), (8, 8, 4), (33, 40, 4), (1000, 1, 3), (2048, 1024, 3),
                                   (2049, 100, 5), (20003, 64, 4), (70001, 1000, 3)])
def test_distill_small(tail, dtype, V, k, n):
    rng = np.random.default_rng(V * 3 + k)
    a = rows_of(rng, n, V, dtype, 2.0)
    t = lists(rng, f64(a, dtype), k, 1.5, tail)
    run_all(a, dtype, t, 1.5, rng.normal(0, 1, n).astype(np.float32))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,V,n", [("bf16", 129280, 3), ("bf16", 131072, 2), ("bf16", 131073, 2), ("f32", 129280, 2),
                                       ("bf16", 129280, 300), ("bf16", 129281, 700), ("f32", 129280, 300), ("f32", 1 << 20, 2),
                                       ("bf16", 140001, 260), ("bf16", 65536, 260), ("f32", 32768, 800), ("f32", 32768, 600), ("bf16", 8192, 3), ("f32", 8193, 3), ("bf16", 32768, 3),
                                       ("f32", 32769, 3)])
def test_distill_long(tail, dtype, V, n):
    """Few rows (split over many workgroups) and many (one or few each)."""
    rng = np.random.default_rng(V + n)
    few = min(n, 8)
    a = rows_of(rng, few, V, dtype, 2.0)
    t = lists(rng, f64(a, dtype), 256, 1.0, tail)
    rep = -(-n // few)
    tile = lambda v: None if v is None else np.concatenate([v] * rep)[:n]
    big = tile(a)
    tt = tuple(tile(v) for v in t)
    w = tile(rng.normal(0, 1, few).astype(np.float32))
    *_, f, g, s = run_all(big, dtype, tt, 1.0, w, rows=list(range(few)) + ([n - 1] if n > few else []))
    for r in range(few, n):  # the copies give the same bits
        assert f["loss"][r] == f["loss"][r % few] and s["loss"][r] == s["loss"][r % few]
    for part in (g, s["grad"]):
        part = part.view(torch.int16 if dtype == "bf16" else torch.int32)
        assert all(torch.equal(part[r], part[r % few]) for r in range(few, n))


@pytest.mark.parametrize("V", [60, 9000, 32768])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_special_student_rows(dtype, tail, V):
    rng = np.random.default_rng(6)
    x = (rng.standard_normal((9, V)) * 2).astype(np.float32)
    x[0, rng.random(V) < 0.5] = -np.inf      # masked vocabulary, part of it on the list: loss +inf
    x[1, :] = -np.inf
    x[1, :4] = [0.5, 1.0, -1.0, 0.0]         # mass on four ids
    x[2, 5:] = -200.0                        # next to none off the first ids
    x[3, :] = 0.0
    x[4, 0] = 90.0                           # all mass on one id
    x[5] -= 1000.0
    x[6] += 1000.0
    x[7, :] = np.float32(-3.3895314e38)
    x[7, 1] = 0.0
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    ids, zl, ln, lse = lists(rng, f64(a, dtype), 5, 1.0, tail, ragged=False)
    ids[1], ids[2] = [0, 1, 2, 3, 9], np.arange(5)
    run_all(a, dtype, (ids, zl, ln, lse), 1.0, np.full(9, 0.5, np.float32))
    # every id off the list is -inf: no mass off it, the last term is left out
    x[0, :] = -np.inf
    x[0, ids[0]] = 1.0
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    run_all(a[:1], dtype, (ids[:1], zl[:1], ln[:1], None if lse is None else lse[:1]), 1.0, np.ones(1, np.float32))


def test_distill_whole_vocabulary_on_the_list():
    rng = np.random.default_rng(12)
    a = rows_of(rng, 3, 512, "f32", 2.0)
    for tail in (False, True):
        t = lists(rng, a.astype(np.float64), 512, 1.0, tail, ragged=False)
        run_all(a, "f32", t, 1.0, np.ones(3, np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 40003])
@pytest.mark.parametrize("temp", [2.0 ** -100, 2.0 ** -10, 2.0 ** 10, 2.0 ** 100])
def test_distill_extreme_temperatures(dtype, V, temp):
    rng = np.random.default_rng(V + 1)
    a = rows_of(rng, 3, V, dtype, 2.0)
    # a teacher's lse keeps 24 bits, which at the lowest temperatures say nothing of its small probabilities
    t = lists(rng, f64(a, dtype), 20, temp, temp >= 1.0)
    run_all(a, dtype, t, temp, np.ones(3, np.float32))


@pytest.mark.parametrize("V", [5003, 32768])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_refused_rows(dtype, V):
    rng = np.random.default_rng(13)
    k, n = 12, 14
    x = (rng.standard_normal((n, V)) * 2).astype(np.float32)
    a = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    t = lists(rng, f64(a, dtype), k, 1.0, True, ragged=False)
    bad = dict(nan=0x7FC0, inf=0x7F80, ninf=0xFF80) if dtype == "bf16" else dict(nan=np.nan, inf=np.inf, ninf=-np.inf)
    exp = np.zeros(n, int)
    t[2][1] = k + 1; exp[1] = L.ST_Q_BAD_LEN
    t[2][2] = -1; exp[2] = L.ST_Q_BAD_LEN
    t[0][3, -1] = V; exp[3] = L.ST_Q_BAD_ID
    t[0][4, 0] = -1; exp[4] = L.ST_Q_BAD_ID
    t[0][5, 3] = t[0][5, 2]; exp[5] = L.ST_Q_UNSORTED
    t[1][6, 4] = np.inf; exp[6] = L.ST_Q_NONFINITE
    t[3][7] = np.nan; exp[7] = L.ST_Q_NONFINITE
    a[8, V - 1] = bad["nan"]; exp[8] = L.ST_ROW_NAN
    a[9, 100] = bad["inf"]; exp[9] = L.ST_ROW_POSINF
    a[10, :] = bad["ninf"]; exp[10] = L.ST_ROW_ZERO_MASS
    a[11, 100] = bad["inf"]; a[11, 4000] = bad["nan"]; exp[11] = L.ST_ROW_NAN
    a[12, :] = bad["nan"]; t[2][12] = 0  # nothing to learn: the row is not read
    a[13, :] = bad["nan"]; t[0][13, 1] = 0; t[0][13, 0] = 1; exp[13] = L.ST_Q_UNSORTED
    for r in range(n):
        s = L.list_status(t[0][r], t[1][r], t[3][r], V, k, int(t[2][r]))
        assert (s or (0 if t[2][r] == 0 else L.row_status(f64(a[r], dtype)))) == exp[r], r
    xd, tt, w = to_dev(a, dtype), teacher(t), torch.ones(n, device=dev())
    f = B.distill(xd, tt)
    g = B.distill_backward(xd, tt, f, w)
    s = B.distill_step(xd, tt, w)
    assert f["status"].tolist() == exp.tolist() and s["status"].tolist() == exp.tolist()
    for r in range(n):
        if exp[r] or t[2][r] == 0:
            assert f["loss"][r] == 0 and s["loss"][r] == 0 and not g[r].any() and not s["grad"][r].any()
    good = [r for r in range(n) if not exp[r]]
    check(a, dtype, t, 1.0, np.ones(n), f["loss"].cpu().numpy(), host64(g), good)
    check(a, dtype, t, 1.0, np.ones(n), s["loss"].cpu().numpy(), host64(s["grad"]), good)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(tail):
    """Central differences of the kernel's own loss.  The loss (near 1) is
    held to 2 D + F < 5e-5 in binary32, so a step of 0.25 sees a slope to 2e-4;
    the third derivative of the loss along one logit is below 0.1 / T^3 q,
    which a step of 0.25 turns into less than 2e-3 of q."""
    rng = np.random.default_rng(15)
    V, h = 64, 0.25
    x = rng.normal(0, 1.0, V).astype(np.float32)
    t = lists(rng, x[None].astype(np.float64), 8, 1.0, tail, ragged=False)
    both = np.stack([x + s * h * np.eye(V, dtype=np.float32)[v] for v in range(V) for s in (1, -1)]).astype(np.float32)
    tt = teacher(tuple(None if v is None else np.repeat(v, 2 * V, 0) for v in t))
    loss = B.distill(to_dev(both, "f32"), tt)["loss"].double().cpu().numpy().reshape(V, 2)
    one = teacher(t)
    grad = host64(B.distill_step(to_dev(x[None], "f32"), one, torch.ones(1, device=dev()))["grad"])[0]
    slope = (loss[:, 0] - loss[:, 1]) / (2 * h)
    assert np.abs(slope - grad).max() < 2e-4 + 2e-3 * 1.0
    assert np.abs(grad).max() > 0.02  # a gradient that the bound tells from nothing


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_in_place_padding_and_strides(dtype):
    rng = np.random.default_rng(16)
    n, V = 6, 4001
    a = rows_of(rng, n, V + 23, dtype, 2.0)
    t = lists(rng, f64(a[:, :V], dtype), 20, 1.0, True)
    tt, w = teacher(t), f32(rng.normal(0, 1, n))
    ref = B.distill_step(to_dev(a[:, :V], dtype), tt, w)
    for how in ("step", "backward"):
        wide = to_dev(a, dtype)
        x, behind = wide[:, :V], wide[:, V:].clone()
        if how == "step":
            s = B.distill_step(x, tt, w, out=x)
            assert torch.equal(s["loss"], ref["loss"])
            got = s["grad"]
        else:
            got = B.distill_backward(x, tt, B.distill(x, tt), w, out=x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(wide[:, V:], behind)
        assert torch.equal(got, ref["grad"]) if how == "step" else True
        check(a[:, :V], dtype, t, 1.0, w.cpu().numpy(), ref["loss"].cpu().numpy(), host64(got))


@pytest.mark.parametrize("V", [700, 32768, 40001])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_bad_logits_on_the_list(dtype, tail, V):
    rng = np.random.default_rng(23)
    x = (rng.standard_normal((4, V)) * 2).astype(np.float32)
    ids, zl, ln, lse = lists(rng, x.astype(np.float64), 9, 1.0, tail, ragged=False)
    x[0, ids[0, 4]] = np.inf
    x[1, ids[1, 8]] = np.nan
    x[2, ids[2, 0]] = np.nan
    x[2, (ids[2, 0] + 1) % V] = np.inf
    a = x if dtype == "f32" else np.where(np.isnan(x), 0x7FC0, W.f32_to_bf16_bits(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf))).astype(np.uint16)
    tt, w = teacher((ids, zl, ln, lse)), torch.ones(4, device=dev())
    f, s = B.distill(to_dev(a, dtype), tt), B.distill_step(to_dev(a, dtype), tt, w)
    exp = [L.ST_ROW_POSINF, L.ST_ROW_NAN, L.ST_ROW_NAN, 0]
    assert f["status"].tolist() == exp and s["status"].tolist() == exp
    assert not f["loss"][:3].any() and not s["grad"][:3].any()
    check(a, dtype, (ids, zl, ln, lse), 1.0, np.ones(4), s["loss"].cpu().numpy(), host64(s["grad"]), [3])


def test_distill_on_two_streams_at_once():
    rng = np.random.default_rng(24)
    n, V = 40, 50001
    cases = []
    for k in (30, 70):
        a = rows_of(rng, n, V, "bf16", 2.0)
        cases.append((to_dev(a, "bf16"), teacher(lists(rng, f64(a, "bf16"), k, 1.0, True)), f32(rng.random(n))))
    ref = [B.distill_step(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for _ in range(20):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                outs.append(B.distill_step(*c))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        for name in ("loss", "grad", "status"):
            assert torch.equal(o[name], ref[i % 2][name]), (i, name)


def test_distill_autograd_captured():
    """Forward and backward of one leaf captured together; no eager graph of that leaf is alive."""
    rng = np.random.default_rng(25)
    n, V = 6, 4001
    a = rows_of(rng, n, V, "f32", 2.0)
    tt, w = teacher(lists(rng, a.astype(np.float64), 20, 1.0, True)), f32(rng.random(n))
    data = to_dev(a, "f32")
    ref = B.distill_step(data, tt, w)
    x = to_dev(a, "f32").requires_grad_()  # (rows that start 16-byte aligned, as data's do)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = B.distill_loss(x, tt)
        (grad,) = torch.autograd.grad(loss, x, w)
    for rep in range(3):
        with torch.no_grad():
            x.copy_(data if rep % 2 == 0 else data + 1.0)  # a shift leaves the softmax as it is
        g.replay()
        torch.cuda.synchronize()
        if rep % 2 == 0:
            assert torch.equal(loss, ref["loss"])
            again = B.distill_backward(data, tt, B.distill(data, tt), w)
            assert torch.equal(grad, again)
        else:
            assert (loss - ref["loss"]).abs().max() < 1e-4 and (grad - ref["grad"]).abs().max() < 1e-5


def test_distill_autograd():
    rng = np.random.default_rng(17)
    n, V = 5, 3000
    a = rows_of(rng, n, V, "f32", 2.0)
    t = lists(rng, a.astype(np.float64), 30, 2.0, True)
    tt = teacher(t)
    x = to_dev(a, "f32").requires_grad_()
    scale = torch.tensor(0.25, device=dev())
    loss = B.distill_loss(x * scale.new_tensor(1.0), tt, 2.0)  # through another operation
    loss.mean().backward()
    check(a, "f32", t, 2.0, np.full(n, 1.0 / n), loss.detach().cpu().numpy(), host64(x.grad))
    # an expanded upstream gradient, and one of another type
    y = to_dev(a, "f32").requires_grad_()
    B.distill_loss(y, tt, 2.0).double().sum().backward()
    check(a, "f32", t, 2.0, np.ones(n), loss.detach().cpu().numpy(), host64(y.grad))
    with pytest.raises(RuntimeError):  # no second derivative
        z = to_dev(a, "f32").requires_grad_()
        (g,) = torch.autograd.grad(B.distill_loss(z, tt, 2.0).sum(), z, create_graph=True)
        g.sum().backward()
    with pytest.raises(RuntimeError):  # the student rows were overwritten between the two passes
        z = to_dev(a, "f32").requires_grad_()
        zz = z * 1.0
        loss = B.distill_loss(zz, tt, 2.0)
        zz.add_(1.0)
        loss.sum().backward()


@pytest.mark.parametrize("how", ["on the host", "float copies", "same place, other stride", "computed again"])
def test_distill_autograd_saved_tensor_hooks(how):
    """What a hook gives back for a saved tensor is what the gradient is computed from."""
    rng = np.random.default_rng(26)
    n, V, wide = 5, 4001 if how == "on the host" else 4000, 4096
    a = rows_of(rng, n, V, "f32", 2.0)
    tt = teacher(lists(rng, a.astype(np.float64), 30, 2.0, True))
    rows = torch.zeros((n, wide), device=dev())
    x = rows[:, :V].copy_(to_dev(a, "f32")).requires_grad_()
    want = B.distill_backward(x.detach(), tt, B.distill(x.detach(), tt, 2.0), torch.ones(n, device=dev()), 2.0)
    if how == "computed again":
        first = {"lse": tt["lse"].clone(), "logits": tt["logits"].clone()}

        def f(y):
            return B.distill_loss(y, dict(tt, lse=first["lse"] * 1.0, logits=first["logits"] * 1.0), 2.0)

        loss = torch.utils.checkpoint.checkpoint(f, x, use_reentrant=False)
        held = [torch.full((n,), -50.0, device=dev()) for _ in range(64)]  # over what the first pass has freed
    else:
        if how == "on the host":
            hooks = torch.autograd.graph.save_on_cpu()
        elif how == "float copies":
            hooks = torch.autograd.graph.saved_tensors_hooks(
                lambda t: t.clone() if t.dtype == torch.float32 and t.shape != x.shape else t, lambda t: t)
        else:
            def unpack(t):
                if t.shape != x.shape:
                    return t
                dense = rows.view(-1)[:n * V].view(n, V)
                return dense.copy_(t)

            hooks = torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone() if t.shape == x.shape else t, unpack)
        with hooks:
            loss = B.distill_loss(x, tt, 2.0)
        if how == "float copies":
            tt["logits"].zero_()
            tt["lse"].zero_()
    (got,) = torch.autograd.grad(loss.sum(), x)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_distill_stream_and_graph_replays():
    rng = np.random.default_rng(18)
    n, V = 4, 9001
    a = rows_of(rng, n, V, "bf16", 2.0)
    tt, w = teacher(lists(rng, f64(a, "bf16"), 50, 1.0, True)), f32(rng.normal(0, 1, n))
    x = to_dev(a, "bf16")

    def both():
        f = B.distill(x, tt)
        s = B.distill_step(x, tt, w)
        return {"loss": f["loss"], "grad": B.distill_backward(x, tt, f, w), "loss2": s["loss"], "grad2": s["grad"]}

    ref = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both()
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both())
        graphs.append(g)
    for rep in range(3):
        for g, o in zip(graphs, outs):
            for v in o.values():
                v.zero_()
            g.replay()
        e = both()
        torch.cuda.synchronize()
        for o in outs + [e, other]:
            for k, v in ref.items():
                assert torch.equal(o[k], v), (rep, k)


def test_distill_far_rows():
    n, V = 16700, 129280
    x = torch.zeros((n, V), dtype=torch.bfloat16, device=dev())
    x[-1, 7] = 4.0
    tt = {"ids": torch.full((n, 1), 7, dtype=torch.int32, device=dev()), "logits": torch.zeros((n, 1), device=dev()),
          "len": torch.ones(n, dtype=torch.int32, device=dev()), "lse": None}
    s = B.distill_step(x, tt, torch.ones(n, device=dev()), out=x)
    want0, want1 = np.log(V), np.log(np.exp(4) + V - 1) - 4
    assert abs(float(s["loss"][0]) - want0) < 1e-4 and abs(float(s["loss"][-1]) - want1) < 1e-4
    assert abs(float(x[-1, 7]) - (np.exp(4) / (np.exp(4) + V - 1) - 1)) < 2.0 ** -8


def test_distill_no_rows():
    x = torch.zeros((0, 64), device=dev())
    tt = {"ids": torch.zeros((0, 4), dtype=torch.int32, device=dev()), "logits": torch.zeros((0, 4), device=dev()),
          "len": torch.zeros(0, dtype=torch.int32, device=dev()), "lse": None}
    f = B.distill(x, tt)
    assert f["loss"].shape == (0,) and B.distill_backward(x, tt, f, torch.zeros(0, device=dev())).shape == (0, 64)
    assert B.distill_step(x, tt, torch.zeros(0, device=dev()))["grad"].shape == (0, 64)
