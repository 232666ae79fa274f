"""Outputs of a beam selection that lie on its inputs, its workspace or each other are refused.  Through the C ABI, with
addresses that are never used: every call here is refused."""
import ctypes

import pytest

from vocab_wide_draft_amd import binding as B

REQUESTS, BEAMS, V, N = 3, 4, 64, 8
STRIDE = 80                                                   # elements of bf16: 32 bytes between rows
ROWS, SCORES, FINISHED, WS = 0x100000, 0x200000, 0x210000, 0x400000
OUT = {"parent": 0x300000, "token": 0x310000, "score": 0x320000, "finished": 0x330000, "len": 0x340000, "status": 0x350000}
BYTES = {name: REQUESTS * (4 if name in ("len", "status") else 4 * N) for name in OUT}


def _message(need_less=0, **at):
    lib = B.load_library()
    rows = B.Rows(ROWS, 1, 0, REQUESTS * BEAMS, V, STRIDE)
    place = {**OUT, "scores": SCORES, "ended": FINISHED, "ws": WS, **at}
    p = {k: ctypes.c_void_p(v) for k, v in place.items()}
    need = lib.dspark_beam_select_workspace(REQUESTS * BEAMS, V, N)
    rc = lib.dspark_beam_select(ctypes.byref(rows), p["scores"], p["ended"], BEAMS, N, 1, p["parent"], p["token"], p["score"],
                                p["finished"], p["len"], p["status"], p["ws"], need - need_less, None)
    assert rc in (-1, -3)
    return lib.dspark_last_error().decode()


def test_places_apart_come_to_the_workspace_check():
    """(No call with a whole workspace is made here: it would start.)"""
    assert "workspace smaller" in _message(need_less=1)


@pytest.mark.parametrize("name", sorted(OUT))
def test_outputs_onto_inputs(name):
    size = BYTES[name]
    reads = {"scores": (SCORES, REQUESTS * BEAMS * 4), "ended": (FINISHED, REQUESTS * BEAMS * 4),
             "rows": (ROWS, (REQUESTS * BEAMS - 1) * STRIDE * 2 + V * 2)}
    for start, bytes_ in reads.values():
        for at in (start, start + bytes_ - 4, start - size + 4):
            assert "overlaps" in _message(**{name: at}), (name, hex(at))
    assert "overlaps" in _message(ws=OUT[name] // 16 * 16)


def test_the_running_scores_in_the_output():
    """The next step's scores in the buffer of this step's."""
    assert "overlaps" in _message(score=SCORES) and "overlaps" in _message(finished=FINISHED)


@pytest.mark.parametrize("name", sorted(OUT))
def test_outputs_onto_each_other(name):
    for other in OUT:
        if other != name:
            assert "overlaps" in _message(**{name: OUT[other]})


def test_a_workspace_onto_inputs():
    for at in (ROWS, SCORES, FINISHED):
        assert "overlaps" in _message(ws=at)
