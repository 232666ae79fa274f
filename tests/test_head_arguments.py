"""Argument checks of the 8-bit head's entry points that return before any device work (through the C ABI, with
addresses that are never used)."""
import ctypes

import pytest
import torch

from vocab_wide_draft_amd import binding as B

fake = ctypes.c_void_p(0x10000)


def _q(n, cols=256, rows=1, kind=0, values=0x10000, scales=0x20000, stride=None, scale_stride=None):
    return B.Fp8(values, scales, kind, rows, n, cols, cols if stride is None else stride,
                 -(-cols // 128) if scale_stride is None else scale_stride)


def _quantize(x, q):
    return B.load_library().dspark_quantize_blocks(ctypes.byref(x), ctypes.byref(q), None)


def test_quantize_refusals():
    x = B.Rows(0x40000, 1, 0, 4, 250, 256)
    for bad in (_q(5), _q(4, 240), _q(4, 272), _q(4, 250), _q(4, 0), _q(4, rows=2), _q(4, kind=2), _q(4, stride=240),
                _q(4, stride=(1 << 22) + 16), _q(4, scale_stride=1), _q(4, values=0), _q(4, scales=0), _q(-1)):
        assert _quantize(x, bad) == -1
    for bad in (_q(4, values=0x10008), _q(4, stride=264), _q(4, scales=0x20002)):
        assert _quantize(x, bad) == -2
    assert _quantize(B.Rows(0x40008, 1, 0, 4, 250, 256), _q(4)) == -2
    assert _quantize(x, _q(4, values=0x40100)) == -1                             # onto the rows
    lib = B.load_library()
    assert lib.dspark_quantize_blocks(None, ctypes.byref(_q(4)), None) == -1
    assert lib.dspark_quantize_blocks(ctypes.byref(x), None, None) == -1
    assert _quantize(B.Rows(None, 1, 0, 0, 250, 256), _q(0, values=0, scales=0)) == 0


def _product(x, w, dt=1, stride=1000, out=0x900000, ws=None, nbytes=0):
    return B.load_library().dspark_block_product(ctypes.byref(x), ctypes.byref(w), ctypes.c_void_p(out), dt, stride, ws, nbytes, None)


def test_product_refusals():
    x, w = _q(4), _q(1000, rows=128)
    assert _product(_q(4, rows=128), w) == -1 and _product(x, _q(1000)) == -1   # a scale for other rows
    assert _product(x, _q(1000, 272, rows=128)) == -1                            # other columns
    assert _product(x, _q(1000, rows=128, kind=1)) == -1                         # other scales
    assert _product(x, w, dt=2) == -1
    assert _product(x, w, stride=999) == -1
    assert _product(x, w, stride=1004) == -2                                     # 2,008 bytes
    assert _product(x, w, out=0x900008) == -2
    assert _product(x, w, out=0) == -1
    assert _product(x, w, out=0x10010) == -1 and _product(_q(4, values=0x800000), _q(1000, rows=128, values=0x900100)) == -1  # onto an input
    assert _product(_q(0), w, out=0) == 0 and _product(x, _q(0, rows=128), out=0) == 0
    lib = B.load_library()
    assert lib.dspark_block_product(None, ctypes.byref(w), fake, 1, 1000, None, 0, None) == -1
    assert lib.dspark_block_product(ctypes.byref(x), None, fake, 1, 1000, None, 0, None) == -1
    # few values from many columns need a workspace
    x, w = _q(4, 20000), _q(40, 20000, rows=128)
    need = lib.dspark_block_product_workspace(4, 40, 20000)
    assert need > 0
    assert _product(x, w, ws=None) == -3 and _product(x, w, ws=fake, nbytes=need - 1) == -3
    assert _product(x, w, ws=ctypes.c_void_p(0x10008), nbytes=need) == -2
    for bad in ((0, 40, 20000), (4, 0, 20000), (4, 40, 0), (4, 40, 1 << 21), (1 << 25, 40, 256), (4, 1 << 25, 256)):
        assert lib.dspark_block_product_workspace(*bad) == 0 and lib.dspark_block_linear_workspace(*bad) == 0


def test_linear_refusals():
    lib = B.load_library()
    x, w = B.Rows(0x40000, 1, 0, 4, 250, 256), _q(1000, rows=128)
    need = lib.dspark_block_linear_workspace(4, 1000, 250)
    assert need >= 4 * 256

    def call(x, w, dt=1, stride=1000, out=0x900000, ws=fake, nbytes=need):
        return lib.dspark_block_linear(ctypes.byref(x), ctypes.byref(w), ctypes.c_void_p(out), dt, stride, ws, nbytes, None)

    assert call(x, _q(1000)) == -1
    assert call(B.Rows(0x40000, 1, 0, 4, 257, 264), w) == -1
    assert call(B.Rows(0x40000, 1, 0, 4, 240, 256), w) == -1
    assert call(B.Rows(0x40000, 3, 0, 4, 250, 256), w) == -1
    assert call(x, w, stride=992) == -1 and call(x, w, stride=1004) == -2 and call(x, w, out=0x900004) == -2
    assert call(x, w, out=0x40010) == -1 and call(x, _q(1000, rows=128, values=0x900100)) == -1
    assert call(x, w, ws=None) == -3 and call(x, w, nbytes=need - 1) == -3
    assert call(x, w, ws=ctypes.c_void_p(0x10004)) == -2
    assert call(B.Rows(None, 1, 0, 0, 250, 256), w, out=0, ws=None, nbytes=0) == 0


def test_transposed_blocks():
    """The transposed head stands for the transpose, on the CPU as on the GPU."""
    v = torch.randn(300, 272).to(torch.float8_e4m3fn)
    s = torch.arange(9.0).reshape(3, 3) + 1
    t = B.transpose_blocks({"values": v, "scales": s}, 260)
    assert t["values"].shape == (260, 304) and t["scales"].shape == (3, 3)
    assert torch.equal(t["values"].float()[:, :300], v.float()[:, :260].t())
    assert not t["values"].float()[:, 300:].any() and torch.equal(t["scales"], s.t())
    with pytest.raises(ValueError):
        B.transpose_blocks({"values": v, "scales": s}, 273)


def test_rows_on_the_cpu_are_refused():
    with pytest.raises(ValueError):
        B.quantize_blocks(torch.zeros(2, 128))
    with pytest.raises(ValueError):
        B.block_linear(torch.zeros(2, 128), {"values": torch.zeros(4, 128).to(torch.float8_e4m3fn), "scales": torch.ones(1, 1)})


def test_scales_apart():
    """Outputs onto scales, and scales onto values or rows, are refused."""
    x = B.Rows(0x40000, 1, 0, 4, 250, 256)
    assert _quantize(x, _q(4, scales=0x40004)) == -1                             # a matrix's scales onto the rows
    assert _quantize(x, _q(4, scales=0x10100)) == -1 and _quantize(x, _q(4, scales=0x0fffc)) == -1  # onto its values
    x, w = _q(4), _q(1000, rows=128, scales=0x30000, values=0x100000)
    assert _product(x, w, out=0x20010) == -1 and _product(x, w, out=0x1fff0) == -1
    assert _product(x, w, out=0x30010) == -1
    rows = B.Rows(0x40000, 1, 0, 4, 250, 256)
    ws = ctypes.c_void_p(0x800000)
    assert B.load_library().dspark_block_linear(ctypes.byref(rows), ctypes.byref(w), ctypes.c_void_p(0x30010), 1, 1000, ws, 1 << 20, None) == -1
