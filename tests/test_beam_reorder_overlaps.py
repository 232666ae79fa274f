"""States that overlap each other are refused, and views that only lie between each other are not.  Through the C ABI with
addresses that are never used: a call whose layouts pass is refused for its missing parents afterwards."""
import ctypes
import random

import pytest

from vocab_wide_draft_amd import binding as B

AT = 1 << 20


def _call(states, requests, beams):
    """None where the layouts pass, otherwise the refusal."""
    lib = B.load_library()
    a = (B.State * len(states))(*states)
    assert lib.dspark_beam_reorder(a, len(states), requests, beams, None, None, None, None) == -1
    message = lib.dspark_last_error().decode()
    return None if message == "NULL parent or req_status" else message


def _state(base, out, strides, outer, rows, row_bytes, to=None):
    return B.State(base, base if out is None else out, *strides, *(strides if to is None else to), outer, rows, row_bytes)


def _refused(states, requests, beams):
    message = _call(states, requests, beams)
    assert message is None or "overlaps another" in message, message
    return message is not None


R, Bm, T, D = 2, 3, 5, 16
PLAIN = (Bm * T * D, T * D, 0, D)
SIZE = R * Bm * T * D


def _plain(base, out=None, **kw):
    return _state(base, out, PLAIN, 1, T, D, **kw)


def test_exchanged_and_shared_states():
    a, b, c, d = (AT + i * SIZE for i in range(4))
    assert not _refused([_plain(a), _plain(b), _plain(c)], R, Bm)                    # one behind the other
    assert not _refused([_plain(a, c), _plain(b, d)], R, Bm)
    assert _refused([_plain(a, b), _plain(b, a)], R, Bm)                             # exchanged
    assert _refused([_plain(a, b), _plain(b, c)], R, Bm)                             # handed on
    assert _refused([_plain(a, c), _plain(b, c)], R, Bm)                             # into one
    assert not _refused([_plain(a, c), _plain(a, d)], R, Bm)                         # out of one
    assert _refused([_plain(a), _plain(a)], R, Bm)
    assert _refused([_plain(a), _plain(a + D)], R, Bm) and _refused([_plain(a + SIZE - 1), _plain(a)], R, Bm)
    # positions 1 .. of the same tensor
    assert _refused([_plain(a), _state(a + D, None, PLAIN, 1, T - 1, D)], R, Bm)
    many = [_plain(AT + i * SIZE) for i in range(300)]
    assert not _refused(many, R, Bm)
    many[299] = _plain(AT + 7 * SIZE + SIZE // 2)
    assert _refused(many, R, Bm)


def test_views_beside_each_other():
    # keys of 24 bytes and values of 16 in positions of 40
    kv = (Bm * T * 40, T * 40, 0, 40)
    keys, values = _state(AT, None, kv, 1, T, 24), _state(AT + 24, None, kv, 1, T, 16)
    assert not _refused([keys, values], R, Bm) and not _refused([values, keys], R, Bm)
    assert _refused([keys, _state(AT + 23, None, kv, 1, T, 16)], R, Bm)
    assert _refused([keys, _state(AT + 24, None, kv, 1, T, 17)], R, Bm)             # the next position's keys
    # layers between beams and positions, whole and with room left behind the positions
    L, H, cap = 4, 3, 7
    layers = [(L * T * D * Bm, L * T * D, 0, D), (Bm * L * H * cap * D, L * H * cap * D, cap * D, D)]
    assert not _refused([_state(AT + i * T * D, None, layers[0], 1, T, D) for i in range(L)], R, Bm)
    heads = [_state(AT + i * H * cap * D, None, layers[1], H, T, D) for i in range(L)]
    assert not _refused(heads, R, Bm)
    assert _refused(heads + [_state(AT + 2 * H * cap * D + (cap - 1) * D, None, layers[1], H, T, D)], R, Bm)
    # positions outermost, beams innermost
    out = (Bm * D, D, 0, R * Bm * D * 2)
    assert not _refused([_state(AT, None, out, 1, T, D), _state(AT + R * Bm * D, None, out, 1, T, D)], R, Bm)


def _bytes(base, strides, sizes, row_bytes):
    at = {base}
    for s, n in zip(strides, sizes):
        at = {x + s * i for x in at for i in range(n)}
    return {x + i for x in at for i in range(row_bytes)}


def _layout(rng, sizes, row_bytes):
    """Nested strides in an order of their own, now and then with room between the parts."""
    reach, strides = row_bytes, [0] * 4
    for k in rng.sample(range(4), 4):
        strides[k] = reach + rng.choice([0, 0, 0, 1, row_bytes, reach, rng.randrange(40)])
        reach = strides[k] * (sizes[k] - 1) + reach if sizes[k] > 1 else reach
    return strides


@pytest.mark.parametrize("seed", range(6))
def test_against_sets_of_bytes(seed):
    rng, met = random.Random(seed), 0
    for _ in range(400):
        r, b = rng.choice([1, 2, 3]), rng.choice([1, 2, 4])
        made, place = [], rng.random() < 0.5
        for _ in range(rng.choice([2, 2, 3])):
            outer, rows, size = rng.choice([1, 2, 3]), rng.choice([0, 1, 3, 6]), rng.randrange(1, 9)
            sizes = (r, b, outer, max(rows, 1))
            strides = list(made[0][0]) if made and rng.random() < 0.5 and made[0][3] == sizes and made[0][4] >= size else _layout(rng, sizes, size)
            base = AT + rng.randrange(0, 400)
            to, out = strides, base
            if not place:
                to, out = _layout(rng, sizes, size), AT + 100000 + rng.randrange(-99600, 400) * rng.choice([0, 1])
            made.append((strides, to, (base, out), sizes, size, outer, rows))
        states = [_state(base, out, s, outer, rows, size, to) for s, to, (base, out), _, size, outer, rows in made]
        reads = [_bytes(m[2][0], m[0], m[3], m[4]) for m in made]
        writes = [_bytes(m[2][1], m[1], m[3], m[4]) for m in made]
        want = any(i != j and writes[i] & (reads[j] | writes[j]) for i in range(len(made)) for j in range(len(made)))
        message = _call(states, r, b)
        if message is not None and "overlaps another" not in message:
            continue  # a state that its own layout has refused
        assert (message is not None) == want
        met += want
    assert met > 20


def test_parents_lengths_and_status():
    """What the call reads of the requests, and the status that it writes, apart from the states and from each other."""
    lib = B.load_library()

    def refused(parent, length, status):
        s = _plain(AT)
        assert lib.dspark_beam_reorder(ctypes.byref(s), 1, R, Bm, parent, length, status, None) == -1
        message = lib.dspark_last_error().decode()
        assert "overlaps another" in message or message == "NULL parent or req_status"
        return "overlaps" in message

    far = AT + 4 * SIZE
    assert refused(AT + 4, None, far) and refused(AT - 4, None, None) and refused(far, AT + SIZE - 4, far + 64)
    assert refused(far, far + 64, AT + 8) and refused(far, None, far + 4 * R * Bm - 4) and refused(far, far + 64, far + 68)
    assert not refused(None, far, far + 4 * R) and not refused(far, far + 4 * R * Bm, None)
