"""Argument checks of the beam search entry points that return before any device work (through the C ABI, with addresses
that are never used), and the plain form against hand-computed steps."""
import ctypes

import numpy as np

from vocab_wide_draft_amd import binding as B

import beam_oracle as O

fake = ctypes.c_void_p(0x10000)


def _select(rows, beams, n_out, end=-1, finished=None, scores=fake, out=fake, ws=fake, nbytes=1 << 30):
    return B.load_library().dspark_beam_select(ctypes.byref(rows), scores, finished, beams, n_out, end, out, out, out, out, out, out,
                                               ws, nbytes, None)


def test_select_refusals():
    r = B.Rows(0x40000, 1, 0, 12, 64, 64)
    for beams, n_out in ((0, 4), (65, 4), (5, 4), (4, 0), (4, 129)):
        assert _select(r, beams, n_out) == -1
    assert _select(B.Rows(0x40000, 1, 0, 64, 64, 64), 64, 65) == -1       # 4,160 in a request
    assert _select(r, 4, 4, end=64) == -1 and _select(r, 4, 4, end=-2) == -1
    assert _select(r, 4, 4, finished=fake) == -1                          # no end_token
    assert _select(r, 4, 4, scores=None) == -1 and _select(r, 4, 4, out=None) == -1
    assert _select(B.Rows(0x40008, 1, 0, 12, 64, 64), 4, 4) == -2
    need = B.load_library().dspark_beam_select_workspace(12, 64, 4)
    assert need > 0
    assert _select(r, 4, 4, ws=None) == -3 and _select(r, 4, 4, nbytes=need - 1) == -3
    assert _select(r, 4, 4, ws=ctypes.c_void_p(0x10008)) == -2
    assert _select(B.Rows(None, 1, 0, 0, 64, 64), 4, 4, scores=None, out=None, ws=None, nbytes=0) == 0
    for bad in ((0, 64, 4), (12, 0, 4), (12, 1 << 21, 4), (12, 64, 0), (12, 64, 129)):
        assert B.load_library().dspark_beam_select_workspace(*bad) == 0


def _state(in_=0x100000, out=None, req=4096, beam=1024, outer=0, row=64, n_outer=1, rows=16, row_bytes=64, **kw):
    s = B.State(in_, in_ if out is None else out, req, beam, outer, row, req, beam, outer, row, n_outer, rows, row_bytes)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _reorder(*states, requests=2, beams=4, parent=fake, st=fake, n=None):
    a = (B.State * max(1, len(states)))(*states)
    return B.load_library().dspark_beam_reorder(a, len(states) if n is None else n, requests, beams, parent, None, st, None)


def test_reorder_refusals():
    assert _reorder(_state(), n=0) == -1
    assert _reorder(_state(), beams=0) == -1 and _reorder(_state(), beams=65) == -1 and _reorder(_state(), requests=-1) == -1
    assert _reorder(_state(), parent=None) == -1 and _reorder(_state(), st=None) == -1
    assert _reorder(_state(in_=0)) == -1
    for bad in (_state(n_outer=0), _state(rows=-1), _state(row_bytes=0), _state(row_bytes=1 << 31), _state(beam=1000),
                _state(req=4000), _state(row=60), _state(beam=0), _state(in_row=128), _state(in_beam=-1024)):
        assert _reorder(bad) == -1
    assert _reorder(_state(rows=1 << 20, row_bytes=1 << 20, row=1 << 20, beam=1 << 41, req=1 << 44)) == -1
    assert _reorder(_state(), _state()) == -1                              # twice
    assert _reorder(_state(), _state(in_=0x200000, out=0x300000)) == -1    # one in place, one not
    assert _reorder(_state(out=0x100000 + 512)) == -1                      # overlaps
    assert _reorder(_state(in_=0, out=0), requests=0, parent=None, st=None) == 0


def test_the_plain_form():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.125, 0.75, 0.125]], np.float32)) + np.float32(3)
    s = np.array([[0.0, -0.5]], np.float32)
    parent, token, score, ended, length, status = O.select(x, s, 4)
    assert parent.tolist() == [[0, 1, 0, 0]] and token.tolist() == [[0, 1, 1, 2]]  # log 0.5, log 0.75 - 0.5, log 0.25 twice
    np.testing.assert_allclose(score, [[np.log(0.5), np.log(0.75) - 0.5, np.log(0.25), np.log(0.25)]], atol=1e-6)
    parent, token, score, ended, length, status = O.select(x, s, 8, np.array([[0, 1]]), 2)
    assert parent.tolist() == [[1, 0, 0, 0, -1, -1, -1, -1]] and token.tolist() == [[2, 0, 1, 2, 0, 0, 0, 0]]
    assert ended.tolist() == [[1, 0, 0, 1, 0, 0, 0, 0]] and length.tolist() == [4]
