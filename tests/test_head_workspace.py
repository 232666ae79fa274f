"""Workspaces of the 8-bit head's calls: those onto an input or the output are refused.  Through the C ABI with addresses
that are never used; every call here is refused."""
import ctypes

from vocab_wide_draft_amd import binding as B

X, XS, W, WS, OUT = 0x100000, 0x200000, 0x1000000, 0x2000000, 0x3000000


def _message(call, ws):
    assert call(ctypes.c_void_p(ws)) == -1
    return B.load_library().dspark_last_error().decode()


def test_onto_inputs_and_outputs():
    lib = B.load_library()
    n, V, cols = 4, 40, 20000
    x, w = B.Fp8(X, XS, 0, 1, n, cols, cols, 157), B.Fp8(W, WS, 0, 128, V, cols, cols, 157)
    rows = B.Rows(X, 1, 0, n, cols, cols)
    need = lib.dspark_block_product_workspace(n, V, cols)
    more = lib.dspark_block_linear_workspace(n, V, cols)
    assert 0 < need < more

    def product(ws):
        return lib.dspark_block_product(ctypes.byref(x), ctypes.byref(w), OUT, 1, V, ws, need, None)

    def linear(ws):
        return lib.dspark_block_linear(ctypes.byref(rows), ctypes.byref(w), OUT, 1, V, ws, more, None)

    places = {X: n * cols, W: V * cols, WS: 157 * 4, OUT: n * V * 2}
    for call, size, own in ((product, need, {**places, XS: n * 157 * 4}), (linear, more, {**places, X: 2 * n * cols})):
        for start, bytes_ in own.items():
            for at in (start, (start + bytes_ - 1) // 16 * 16, (start - size) // 16 * 16 + 16):
                assert "workspace overlaps" in _message(call, at), hex(at)


def test_a_workspace_of_more_rows_serves_fewer():
    lib = B.load_library()
    rows = [*range(1, 700), *range(700, 6000, 29), 1 << 16, 1 << 24]
    for N, K in ((150, 9000), (1, 1 << 20), (5120, 129280), (640, 1 << 20), (1000, 3000), (27489, 28027), (129280, 5120), (20003, 1000)):
        for query in (lib.dspark_block_product_workspace, lib.dspark_block_linear_workspace):
            sizes = [query(n, N, K) for n in rows]
            assert sizes == sorted(sizes)


def test_a_workspace_of_a_few_dozen_rows_serves_fewer():
    """Lengths of w for which 17 to 32 rows, too, are taken in tiles."""
    lib = B.load_library()
    for N, K in ((98253, 3120), (1000, 125000), (640, 300000), (12000, 20000), (40000, 5120), (300, 1 << 19), (2000, 150000)):
        for query in (lib.dspark_block_product_workspace, lib.dspark_block_linear_workspace):
            sizes = [query(n, N, K) for n in range(1, 130)]
            assert sizes == sorted(sizes)
