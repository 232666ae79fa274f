"""Argument checks of the logit operators that return before any device
work (through the C ABI, with addresses that are never used)."""
import ctypes

import pytest
import torch

from vocab_wide_draft_amd import binding as B

fake = ctypes.c_void_p(0x10000)


def _shape(rows, how, out=0x900000, dt=1, stride=64, st=fake):
    return B.load_library().dspark_shape_logits(ctypes.byref(rows), ctypes.byref(how), ctypes.c_void_p(out), dt, stride,
                                                st, None)


def _how(P=1, **kw):
    h = B.Shaping()
    h.rows_per_request = P
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def test_shape_refusals():
    r = B.Rows(0x10000, 1, 0, 6, 64, 64)
    assert _shape(r, _how(0)) == -1
    assert _shape(r, _how(4)) == -1                                       # 6 rows, 4 a request
    assert _shape(r, _how(), dt=5) == -1
    assert _shape(B.Rows(0x10000, 0, 0, 6, 64, 64), _how(), dt=1) == -1   # float32 rows to bf16
    assert _shape(r, _how(), stride=63) == -1
    assert _shape(r, _how(), stride=68) == -2                             # 136 bytes
    assert _shape(r, _how(), out=0x900008) == -2
    assert _shape(r, _how(), out=0x10000, dt=0) == -1                     # in place with another type
    assert _shape(r, _how(), out=0x10000, stride=72) == -1                # in place with another stride
    assert _shape(r, _how(), out=0x10080) == -1                           # overlaps
    assert "overlap" in B.load_library().dspark_last_error().decode()
    assert _shape(r, _how(), out=0x10000 - 128 * 5) == -1
    assert _shape(r, _how(), out=0) == -1
    assert _shape(r, _how(), st=None) == -1
    assert _shape(r, _how(history=1, history_max=8, history_stride=7)) == -1
    assert _shape(r, _how(history=1, history_max=-1, history_stride=7)) == -1
    assert _shape(r, _how(history=1, history_max=(1 << 30) + 1, history_stride=1 << 31)) == -1
    assert _shape(r, _how(history=1, history_max=8, history_stride=8)) == -1  # no history_len
    assert _shape(r, _how(6, draft=1, draft_stride=4)) == -1
    assert _shape(r, _how(bias_offset=1, bias_total=-1)) == -1
    assert _shape(r, _how(bias_offset=1, bias_total=4)) == -1             # no ids
    assert _shape(r, _how(mask=1, mask_stride=1, n_masks=6)) == -1        # 64 ids need two words
    assert _shape(r, _how(mask=1, mask_stride=2, n_masks=5)) == -1        # fewer masks than rows
    assert B.load_library().dspark_shape_logits(ctypes.byref(r), None, fake, 1, 64, fake, None) == -1
    assert _shape(B.Rows(None, 1, 0, 0, 64, 64), _how(6), out=0, st=None) == 0


def _top(rows, k, temp=1.0, ids=fake, ln=fake):
    return B.load_library().dspark_top_logits(ctypes.byref(rows), None, k, temp, ids, fake, ln, None, fake, None, 0, None)


def test_top_refusals():
    r = B.Rows(0x10000, 1, 0, 6, 64, 64)
    assert _top(r, -1) == -1
    assert _top(r, 1025) == -1
    for t in (0.0, -1.0, float("inf"), float("nan"), 1e-45, 2.0 ** -101, 2.0 ** 101):
        assert _top(r, 4, t) == -1, t
    assert _top(r, 4, ids=None) == -1
    assert _top(r, 4, ln=None) == -1
    assert _top(B.Rows(0x10008, 1, 0, 6, 64, 64), 4) == -2
    assert _top(B.Rows(None, 1, 0, 0, 64, 64), 4, ids=None, ln=None) == 0


def test_distill_refusals():
    lib = B.load_library()
    r = B.Rows(0x100000, 1, 0, 6, 64, 64)
    V = 65536
    r = B.Rows(0x100000, 1, 0, 6, V, V)  # long enough for a workspace in every entry point
    need = lib.dspark_distill_workspace(6, V)
    assert lib.dspark_distill_workspace(6, 64) == 0  # short rows need none
    assert need > 0 and lib.dspark_distill_workspace(0, V) == 0 and lib.dspark_distill_workspace(6, 0) == 0
    t = B.Teacher(0x10000, 0x10000, 0x10000, None, 8, 0)

    def fwd(r=r, t=t, T=1.0, loss=fake, ws=0x40000, n=need):
        return lib.dspark_distill(ctypes.byref(r), ctypes.byref(t), T, loss, fake, fake, ctypes.c_void_p(ws), n, None)

    def bwd(r=r, t=t, T=1.0, st=fake, grad=0x900000, stride=65536):
        return lib.dspark_distill_backward(ctypes.byref(r), ctypes.byref(t), T, st, fake, fake, ctypes.c_void_p(grad),
                                           stride, None)

    def step(r=r, t=t, T=1.0, w=fake, grad=0x900000, stride=65536, ws=0x40000, n=need):
        return lib.dspark_distill_step(ctypes.byref(r), ctypes.byref(t), T, w, fake, ctypes.c_void_p(grad), stride, fake,
                                       ctypes.c_void_p(ws), n, None)

    bad_t = [B.Teacher(0x10000, 0x10000, 0x10000, None, 1025, 0), B.Teacher(0x10000, 0x10000, 0x10000, None, -1, 0),
             B.Teacher(None, 0x10000, 0x10000, None, 8, 0), B.Teacher(0x10000, 0x10000, None, None, 8, 0)]
    for f in (fwd, bwd, step):
        for x in bad_t:
            assert f(t=x) == -1
        assert f(T=0.0) == -1 and f(T=float("nan")) == -1
        assert f(r=B.Rows(0x100000, 1, 0, 6, V, V + 4)) == -2
    assert fwd(loss=None) == -1 and bwd(st=None) == -1 and step(w=None) == -1
    for f in (fwd, step):
        assert f(n=need - 1) == -3 and f(ws=0) == -3 and f(ws=0x40008) == -2
    for f in (bwd, step):
        assert f(grad=0x900008) == -2 and f(stride=V - 1) == -1 and f(grad=0) == -1
        assert f(grad=0x100080) == -1                          # overlaps the student rows
        assert f(grad=0x100000, stride=V + 8) == -1               # in place with another stride
    empty = B.Rows(None, 1, 0, 0, 64, 64)
    t0 = B.Teacher(None, None, None, None, 8, 0)
    assert fwd(r=empty, t=t0, loss=None, ws=0, n=0) == 0 and bwd(r=empty, t=t0, st=None, grad=0) == 0
    assert step(r=empty, t=t0, w=None, grad=0, ws=0, n=0) == 0


def test_workspaces_grow_with_the_rows():
    """One workspace for the largest batch serves every smaller one."""
    lib = B.load_library()
    ns = list(range(1, 300)) + [511, 512, 513, 1000, 2047, 2048, 2049, 5120, 1 << 20, 1 << 24]
    for V in (1, 2048, 8000, 16384, 16385, 32768, 32769, 40000, 65536, 65537, 129280, 131072, 131073, 200000, 1 << 20):
        for k in (0, 1, 64, 1024):
            sizes = [lib.dspark_top_logits_workspace(n, V, k) for n in ns]
            assert sizes == sorted(sizes), (V, k)
        sizes = [lib.dspark_distill_workspace(n, V) for n in ns]
        assert sizes == sorted(sizes), V


def test_binding_refuses_wrong_tensors():
    dev = torch.device("cpu")
    with pytest.raises(ValueError):
        B._arg(torch.zeros(3, dtype=torch.int64), "x", torch.int32, (3,), dev)
    with pytest.raises(ValueError):
        B._arg(torch.zeros(4, dtype=torch.int32), "x", torch.int32, (3,), dev)
    with pytest.raises(ValueError):
        B._arg(torch.zeros(6, dtype=torch.int32)[::2], "x", torch.int32, (3,), dev)
    with pytest.raises(ValueError):
        B._matrix(torch.zeros((4, 3), dtype=torch.int32).t(), "x", torch.int32, 3, dev)
    with pytest.raises(ValueError):
        B._matrix(torch.zeros((1, 3), dtype=torch.int32).expand(2, 3), "x", torch.int32, 2, dev)
    a, cols, stride = B._matrix(torch.zeros((3, 8), dtype=torch.int32)[:, :5], "x", torch.int32, 3, dev)
    assert (cols, stride) == (5, 8)
    t = {"ids": torch.zeros((2, 3), dtype=torch.int32), "logits": torch.zeros((2, 3), requires_grad=True),
         "len": torch.zeros(2, dtype=torch.int32), "lse": None}
    with pytest.raises(ValueError):
        B.distill_loss(torch.zeros((2, 8)), t)
    for call in (lambda x: B.shape_logits(x), lambda x: B.top_logits(x, 1), lambda x: B.distill(x, t)):
        with pytest.raises(ValueError):
            call(torch.zeros((2, 8)))  # rows not on the GPU
