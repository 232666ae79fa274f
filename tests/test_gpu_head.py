"""Quantisation in blocks and the 8-bit head's product and gradient against numpy and torch in 64 bits.

Tolerances.  Quantised values and scales are exact.  The product of the quantised matrices is exact for each pair (4 by 4
significant bits); K of them and K / 128 scales are added and multiplied in binary32, each sum off by at most
(K + 2 K / 128 + 4) 2^-24 of the sum of the products' absolute values however it is ordered.  For bf16 results each
product is cut to 2^-13 of the largest of its eight neighbours (off by up to 7 * 2^-13 of the sum of the eight), and the
sum is rounded by another 2^-8 of itself."""
import numpy as np
import pytest
import torch

from vocab_wide_draft_amd import binding as B

from head_oracle import KINDS, e4m3, quantize, wide, worth

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _x(n, width, dtype, seed, spread=2.0):
    g = _gen(seed)
    x = torch.randn((n, width), generator=g) * torch.exp(spread * torch.randn((n, 1), generator=g))
    return x.to(dtype)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("n,width", [(1, 1), (1, 128), (3, 127), (5, 129), (130, 300), (257, 2500), (7, 5120)])
def test_quantize(n, width, rows, dtype, kind):
    x = _x(n, width, dtype, 100 * n + width)
    if n > 2:
        x[1] = 0
        x[2, : min(width, 128)] = 1.75 * 2.0 ** 20  # 448 times a power of two, the border of the next
        x[0] *= 2.0 ** -60
    q = B.quantize_blocks(wide(x, dev), rows, KINDS[kind])
    values, scales = quantize(x.float().numpy(), rows, kind == "pow2")
    assert q["values"].shape == values.shape and q["scales"].shape == scales.shape
    assert np.array_equal(q["scales"].float().cpu().double().numpy(), scales)
    assert np.array_equal(q["values"].float().cpu().double().numpy(), values)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
def test_quantize_every_step(kind):
    """Quotients at, and next to, each border between two values of e4m3, and below the smallest."""
    grid = np.unique(e4m3(np.linspace(-448, 448, 400001)))
    small = np.ldexp(np.arange(-40, 41), -12)
    y = np.unique(np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, small])).astype(np.float32)
    y = np.unique(np.concatenate([y, np.nextafter(y, np.float32(1e9)), np.nextafter(y, np.float32(-1e9))]))
    y = y[np.abs(y) <= 448]
    blocks = -(-y.size // 127)
    x = np.zeros((blocks, 128), np.float32)
    x[:, 0] = 448  # scale 1
    x[:, 1:].reshape(-1)[: y.size] = 0
    for i in range(blocks):
        part = y[127 * i:127 * (i + 1)]
        x[i, 1:1 + part.size] = part
    q = B.quantize_blocks(torch.from_numpy(x).to(dev), 1, KINDS[kind])
    assert (q["scales"].float() == 1).all()
    assert np.array_equal(q["values"].float().cpu().double().numpy(), e4m3(x))


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_extremes(rows, kind):
    x = torch.zeros(140, 640)
    x[0, :128] = torch.linspace(-3.4e38, 3.4e38, 128)
    x[3, 128:256] = 1e-45      # subnormal: the least scale
    x[5, 256] = float("inf")
    x[6, 384] = float("nan")
    x[139, 520] = -float("inf")
    x[138, 520] = 5.0
    q = B.quantize_blocks(x.to(dev), rows, KINDS[kind])
    values, scales = quantize(x.numpy(), rows, kind == "pow2")
    np.testing.assert_array_equal(q["scales"].float().cpu().double().numpy(), scales)
    np.testing.assert_array_equal(q["values"].float().cpu().double().numpy(), values)
    assert np.isnan(scales).any()


def test_quantize_leaves_the_rest_alone():
    """Rows inside wider buffers: nothing outside them is read or written."""
    big = torch.full((9, 512), float("nan"), device=dev)
    x = big[2:7, 64:264]
    x.copy_(_x(5, 200, torch.float32, 3))
    out = torch.full((9, 512), 7, dtype=torch.uint8, device=dev)
    v = out[2:7, 64:272].view(torch.float8_e4m3fn)
    s = torch.full((9, 16), 5.0, device=dev)
    q = {"values": v, "scales": s[2:7, 4:6]}
    import ctypes
    r, f = B._rows(x), B._fp8(q, "out", 1, dev)
    B._check(B.load_library().dspark_quantize_blocks(ctypes.byref(r), ctypes.byref(f), B._stream()))
    values, scales = quantize(x.cpu().numpy(), 1, False)
    assert np.array_equal(v.float().cpu().double().numpy(), values)
    assert np.array_equal(s[2:7, 4:6].cpu().double().numpy(), scales)
    out[2:7, 64:272] = 7
    s[2:7, 4:6] = 5.0
    assert (out == 7).all() and (s == 5.0).all()


def _weight(V, width, kind, seed):
    return B.quantize_blocks(wide(_x(V, width, torch.float32, seed, 0.5), dev), 128, KINDS[kind])


def _check(got, x, w, dtype):
    """got [n, V] against the 64-bit product of x and w (as 64-bit matrices)."""
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    K = x.shape[1]
    tol = size * ((K + 2 * (K // 128 + 1) + 4) * 2.0 ** -24)
    if dtype == torch.bfloat16:
        tol = tol + size * (7 * 2.0 ** -13)
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    off = (got.cpu().double() - want).abs()
    assert (off <= tol).all(), float((off / tol).max())


SIZES = [(1, 1, 1), (1, 17, 128), (2, 130, 129), (15, 260, 256), (16, 257, 640), (17, 300, 1000), (33, 64, 2064),
         (64, 513, 384), (65, 500, 500), (128, 128, 128), (129, 385, 272), (300, 700, 1296), (513, 1030, 512)]


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V,width", SIZES)
def test_product(n, V, width, out, kind):
    x = B.quantize_blocks(wide(_x(n, width, torch.bfloat16, n + V), dev), 1, KINDS[kind])
    w = _weight(V, width, kind, n * V + 1)
    _check(B.block_product(x, w, out), worth(x, 1), worth(w, 128), out)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("n,V,width", SIZES + [(40, 300, 20000), (2, 129280, 256)])
def test_product_of_whole_numbers_is_exact(n, V, width, kind):
    """Small whole numbers, whose products and sums no step has to round; sums that bf16 holds."""
    cols, g = -(-width // 16) * 16, _gen(n * V)
    few = min(1.0, 100.0 / width)
    x = torch.randint(-1, 2, (n, cols), generator=g).float() * (torch.rand((n, cols), generator=g) < few)
    w = torch.randint(-2, 3, (V, cols), generator=g).float()
    sx = 2.0 ** torch.randint(-3, 4, (n, -(-cols // 128)), generator=g).float()
    sw = torch.ones(-(-V // 128), -(-cols // 128)) * 2.0 ** torch.randint(-3, 4, (-(-V // 128), 1), generator=g).float()
    sx[:] = sx[:, :1]
    q = [{"values": v.to(dev).to(torch.float8_e4m3fn), "scales": s.to(dev).to(KINDS[kind])} for v, s in ((x, sx), (w, sw))]
    want = (x.to(dev).double() @ w.to(dev).double().t())
    assert want.abs().max() <= 256
    want = want * sx[:, :1].to(dev).double() * sw[:, 0].repeat_interleave(128)[:V].to(dev).double()
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(B.block_product(*q, out).double(), want)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("n,V,width", [(1, 40, 20003), (5, 200, 30000), (40, 128, 16400), (200, 150, 9000)])
def test_product_of_long_rows(n, V, width, kind):
    """Few output values and many columns, as in the gradient: the columns are split."""
    x = B.quantize_blocks(wide(_x(n, width, torch.float32, 7), dev), 1, KINDS[kind])
    w = _weight(V, width, kind, 8)
    for out in (torch.float32, torch.bfloat16):
        _check(B.block_product(x, w, out), worth(x, 1), worth(w, 128), out)


@pytest.mark.parametrize("n", [1, 16, 24, 32, 33, 64, 384])
def test_product_of_a_full_vocabulary(n):
    V, width = 129280, 1024
    x = B.quantize_blocks(_x(n, width, torch.bfloat16, 5).to(dev), 1)
    w = _weight(V, width, "f32", 6)
    _check(B.block_product(x, w, torch.bfloat16), worth(x, 1), worth(w, 128), torch.bfloat16)


@pytest.mark.parametrize("n", [1, 20, 100])
def test_offsets_beyond_32_bits(n):
    """A head of more than 4 GiB: its last rows are the right ones."""
    V, width = (1 << 32) // 4096 + 300, 4096
    values = torch.zeros((V, width), dtype=torch.float8_e4m3fn, device=dev)
    w = {"values": values, "scales": torch.ones((-(-V // 128), width // 128), device=dev)}
    part = e4m3(_x(400, width, torch.float32, 3, 0.1).numpy().clip(-4, 4))
    values[-400:] = torch.from_numpy(part).to(dev).to(torch.float8_e4m3fn)
    x = B.quantize_blocks(_x(n, width, torch.bfloat16, 4).to(dev), 1)
    got = B.block_product(x, w, torch.float32)
    _check(got[:, -400:], worth(x, 1), torch.from_numpy(part), torch.float32)
    assert not got[:, :-400].any()


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("n,V,width", [(3, 200, 300), (70, 300, 512)])
def test_strides_and_what_lies_between_rows(n, V, width, kind):
    cols = -(-width // 16) * 16
    vals = torch.full((n, cols + 48), 0x7F, dtype=torch.uint8, device=dev)   # NaN between the rows
    wvals = torch.full((V, cols + 32), 0x7F, dtype=torch.uint8, device=dev)
    xq = B.quantize_blocks(wide(_x(n, width, torch.bfloat16, 1), dev), 1, KINDS[kind])
    wq = _weight(V, width, kind, 2)
    vals[:, :cols] = xq["values"].view(torch.uint8)
    wvals[:, 16:cols + 16] = wq["values"].view(torch.uint8)
    sx = torch.full((n, xq["scales"].shape[1] + 3), float("nan"), device=dev).to(KINDS[kind])
    sx[:, 1:1 + xq["scales"].shape[1]] = xq["scales"]
    x = {"values": vals[:, :cols].view(torch.float8_e4m3fn), "scales": sx[:, 1:1 + xq["scales"].shape[1]]}
    w = {"values": wvals[:, 16:cols + 16].view(torch.float8_e4m3fn), "scales": wq["scales"]}
    out = torch.full((n, -(-V // 8) * 8 + 24), 3.0, device=dev)
    B.block_product(x, w, torch.float32, out=out[:, :V])
    assert torch.equal(out[:, :V], B.block_product(xq, wq, torch.float32))
    assert (out[:, V:] == 3.0).all()


def test_rows_do_not_depend_on_their_neighbours():
    """The rows of a batch that the same kernel takes, shifted, give the same bits; and so does a second call."""
    w = _weight(700, 1024, "f32", 2)
    x = _x(100, 1024, torch.bfloat16, 1).to(dev)
    a = B.block_linear(x, w)
    assert torch.equal(a, B.block_linear(x, w))
    assert torch.equal(B.block_linear(x.flip(0).contiguous(), w).flip(0), a)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
def test_nan_and_infinity_reach_their_row(kind):
    w = _weight(300, 400, kind, 2)
    x = _x(20, 400, torch.bfloat16, 1)
    x[3, 17], x[7, 399], x[9, 130] = float("nan"), float("inf"), -float("inf")
    y = B.block_linear(wide(x, dev), w, torch.float32)
    bad = torch.zeros(20, dtype=torch.bool, device=dev)
    bad[[3, 7, 9]] = True
    assert y[bad].isnan().all() and y[~bad].isfinite().all()
    assert B.propose(wide(y.cpu(), dev))["status"].tolist() == [int(b) for b in bad]  # ROW_NAN


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("n,V", [(3, 700), (40, 300), (200, 500)])
def test_nan_scales(n, V, kind):
    """A scale that is a NaN reaches the outputs of its rows, and no others, whatever its values are."""
    x = B.quantize_blocks(_x(n, 512, torch.bfloat16, 1).to(dev), 1, KINDS[kind])
    w = _weight(V, 512, kind, 2)
    sx, sw = x["scales"].float(), w["scales"].float()
    sx[n // 2, 2] = float("nan")
    sw[1, 3] = float("nan")
    bad = torch.zeros((n, V), dtype=torch.bool, device=dev)
    bad[n // 2] = True
    bad[:, 128:256] = True
    q = [{"values": t["values"], "scales": s.to(KINDS[kind])} for t, s in ((x, sx), (w, sw))]
    for out in (torch.float32, torch.bfloat16):
        y = B.block_product(*q, out)
        assert y[bad].isnan().all() and y[~bad].isfinite().all()


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V,width", [(1, 300, 500), (5, 1000, 512), (16, 2000, 130), (40, 333, 1024), (150, 700, 256)])
def test_linear_is_quantisation_and_product(n, V, width, dtype, kind):
    w = _weight(V, width, kind, 2)
    x = wide(_x(n, width, dtype, 1), dev)
    q = B.quantize_blocks(x, 1, KINDS[kind])
    for out in (torch.float32, torch.bfloat16):
        _check(B.block_linear(x, w, out), worth(q, 1), worth(w, 128), out)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V,width", [(1, 300, 200), (6, 1500, 512), (50, 2003, 129), (140, 640, 384)])
def test_gradient(n, V, width, dtype, kind):
    """The gradient is the quantised gradient of the logits times what the head stands for."""
    weight = _weight(V, width, kind, 2)
    head = {"weight": weight, "transposed": B.transpose_blocks(weight, width)}
    assert torch.equal(worth(head["transposed"], 128)[:, :V], worth(weight, 128)[:, :width].t())
    x = wide(_x(n, width, dtype, 1), dev).requires_grad_()
    y = B.head_logits(x, head)
    assert torch.equal(y, B.block_linear(x.detach(), weight)) and y.dtype == dtype
    up = wide(_x(n, V, dtype, 9), dev)
    (dx,) = torch.autograd.grad(y, x, up)
    assert dx.shape == x.shape and dx.dtype == dtype
    g = worth(B.quantize_blocks(up, 1, KINDS[kind]), 1)[:, :V].contiguous()
    _check(dx, g, worth(weight, 128)[:, :width].t().contiguous(), dtype)


@pytest.mark.parametrize("kind", ["f32", "pow2"])
def test_gradient_against_differences(kind):
    """sum(up * logits) along a direction, between hidden states that e4m3 holds exactly: the logits are linear there.
    A gradient quantised to e4m3 is off by 2^-4 of itself, or 2^-10 of its block's scale where it is small."""
    n, V, width = 6, 900, 256
    weight = _weight(V, width, kind, 2)
    head = {"weight": weight, "transposed": B.transpose_blocks(weight, width)}
    g = _gen(4)
    x = torch.randint(-8, 9, (n, width), generator=g).float()
    d = torch.randint(-4, 5, (n, width), generator=g).float()
    x[:, ::128], d[:, ::128] = 448.0, 0.0  # scales of 1, so that x, x + d and x - d are held exactly
    x, d = x.to(dev), d.to(dev)
    up = torch.randn((n, V), generator=g).to(dev)
    up_wide = wide(up.cpu(), dev)
    at = x.clone().requires_grad_()
    (dx,) = torch.autograd.grad(B.head_logits(at, head), at, up_wide)
    hi, lo = (B.head_logits(x + s * d, head).double() for s in (1, -1))
    slope = ((hi - lo) / 2 * up.double()).sum(1)
    W = worth(weight, 128).to(dev)[:, :width]
    s = B.quantize_blocks(up_wide, 1, KINDS[kind])["scales"].float().double().repeat_interleave(128, 1)[:, :V]
    off = torch.maximum(up.double().abs() * 2.0 ** -4, s * 2.0 ** -10)
    lin = (d.double() @ W.t()).abs()
    sums = (x.double().abs() + d.double().abs()) @ W.abs().t() * ((width + 12) * 2.0 ** -24)
    tol = (off * lin).sum(1) + (sums * up.double().abs()).sum(1) + (dx.double() * d.double()).abs().sum(1) * (V + 40) * 2.0 ** -24
    assert ((dx.double() * d.double()).sum(1) - slope).abs().le(tol).all()


def test_gradient_of_expanded_and_sliced():
    """Gradients that are no rows of their own: one value for all, every second column, a transposed matrix."""
    weight = _weight(300, 256, "pow2", 2)
    head = {"weight": weight, "transposed": B.transpose_blocks(weight, 256)}
    x = _x(9, 256, torch.float32, 1).to(dev).requires_grad_()
    ones = torch.ones((9, 304), device=dev)[:, :300]
    (want,) = torch.autograd.grad(B.head_logits(x, head), x, ones)
    (got,) = torch.autograd.grad(B.head_logits(x, head).sum(), x)
    assert torch.equal(got, want)
    t = torch.randn((300, 9), device=dev)
    (want,) = torch.autograd.grad(B.head_logits(x, head), x, wide(t.t().cpu().contiguous(), dev))
    (got,) = torch.autograd.grad(B.head_logits(x, head), x, t.t())
    assert torch.equal(got, want)


def test_second_derivative_is_refused():
    weight = _weight(300, 256, "pow2", 2)
    head = {"weight": weight, "transposed": B.transpose_blocks(weight, 256)}
    x = _x(4, 256, torch.float32, 1).to(dev).requires_grad_()
    (dx,) = torch.autograd.grad(B.head_logits(x, head).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_no_rows():
    weight = _weight(300, 256, "f32", 2)
    x = torch.empty((0, 256), device=dev)
    assert B.block_linear(x, weight).shape == (0, 300)
    q = B.quantize_blocks(x)
    assert q["values"].shape == (0, 256) and B.block_product(q, weight).shape == (0, 300)


@pytest.mark.parametrize("n", [1, 30, 200])
def test_streams_and_graphs(n):
    """On another stream than the tensors' own, two calls at once, and captured and replayed with other inputs."""
    weight = _weight(1000, 3000, "f32", 2)
    a, b = (_x(n, 3000, torch.bfloat16, k).to(dev) for k in (1, 2))
    want = B.block_linear(a, weight), B.block_linear(b, weight)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        y1 = [B.block_linear(a, weight) for _ in range(5)]
    with torch.cuda.stream(s2):
        y2 = [B.block_linear(b, weight) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[0]) for y in y1) and all(torch.equal(y, want[1]) for y in y2)
    x = a.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = B.block_linear(x, weight)
    for k in (1, 0, 1):
        x.copy_((a, b)[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k])
        B.block_linear(b, weight)


def test_refusals():
    w = _weight(300, 256, "f32", 2)
    x = torch.zeros((4, 256), device=dev)
    with pytest.raises(ValueError):
        B.block_linear(x, {"values": w["values"], "scales": w["scales"][:2]})
    with pytest.raises(ValueError):
        B.block_linear(x, {"values": w["values"].view(torch.uint8), "scales": w["scales"]})
    with pytest.raises(B.DsparkError):
        B.block_linear(torch.zeros((4, 200), device=dev), w)
    with pytest.raises(B.DsparkError):
        B.block_linear(torch.zeros((4, 300), device=dev)[:, 1:257], w)  # unaligned rows
    with pytest.raises(B.DsparkError):
        B.block_product(B.quantize_blocks(x, 1, torch.float8_e8m0fnu), w)  # scales of two types
    with pytest.raises(ValueError):
        B.head_logits(x.requires_grad_(), {"weight": w})
    with pytest.raises(ValueError):
        B.quantize_blocks(x.detach(), 64)
