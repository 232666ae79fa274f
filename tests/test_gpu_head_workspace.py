"""A workspace of the 8-bit head's product that was made for a batch serves every smaller one, and the products in it are
those in workspaces of their own, bit for bit."""
import ctypes

import pytest
import torch

from vocab_wide_draft_amd import binding as B

from head_oracle import KINDS

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("most,V,width", [(2900, 150, 9008), (1100, 40, 20000), (700, 5120, 32768)])
def test_one_workspace_for_all_batches(most, V, width, kind):
    lib = B.load_library()
    g = torch.Generator(device=dev).manual_seed(most)
    x = torch.randn((most, width), generator=g, device=dev).to(torch.bfloat16)
    w = B.quantize_blocks(torch.randn((V, width), generator=g, device=dev), 128, KINDS[kind])
    fw = B._fp8(w, "w", 128, dev)
    stride = B._padded(V, torch.bfloat16)
    need = lib.dspark_block_product_workspace(most, V, width), lib.dspark_block_linear_workspace(most, V, width)
    ws = torch.empty(max(need), dtype=torch.uint8, device=dev)
    for n in (most, 640, 320, 257, 256, 129, 65, 64, 33, 32, 17, 16, 1):
        q = B.quantize_blocks(x[:n], 1, KINDS[kind])
        want = B.block_product(q, w)
        rows, fx = B._rows(x[:n]), B._fp8(q, "x", 1, dev)
        for way in ("product", "linear"):
            out = torch.zeros((n, stride), dtype=torch.bfloat16, device=dev)
            ws.fill_(0xFF)  # NaN
            if way == "product":
                rc = lib.dspark_block_product(ctypes.byref(fx), ctypes.byref(fw), out.data_ptr(), 1, stride, ws.data_ptr(), need[0], B._stream())
            else:
                rc = lib.dspark_block_linear(ctypes.byref(rows), ctypes.byref(fw), out.data_ptr(), 1, stride, ws.data_ptr(), need[1], B._stream())
            assert rc == 0, (n, way, lib.dspark_last_error())
            assert torch.equal(out[:, :V], want), (n, way)
