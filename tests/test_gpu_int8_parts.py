"""8-bit integer products whose sums are computed in parts, against float64
products of the codes (exact) on the GPU, bit for bit; that the products of the
list are in parts is checked without one."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from int8_util import DT
from test_gpu_int8_tiles import product, tables

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

# M, N, rows: small products found for each kind of tile, from few parts to many
PARTS = {"32 x 64": [(5654, 5342, 28), (720, 4207, 177), (183, 2971, 165), (17, 3128, 33), (16, 4691, 5), (16, 5703, 1)],
         "64 x 64": [(583, 5123, 411), (230, 3804, 404), (107, 3220, 397), (168, 6452, 161), (37, 6094, 322)],
         "64 x 128": [(553, 8951, 1552), (723, 5694, 483), (693, 8421, 213), (455, 12565, 211), (558, 14363, 76), (497, 16136, 88)],
         "128 x 64": [(1218, 10681, 1291), (616, 6691, 902), (870, 8294, 420), (331, 11994, 677), (365, 19858, 424)],
         "128 x 128": [(1146, 10823, 1396), (732, 6408, 735), (1024, 8192, 700), (449, 9331, 732), (329, 13956, 709), (485, 19819, 325)]}
LIST = [c for cases in PARTS.values() for c in cases]
OUT = {"f32": sk.F32, "bf16": sk.BF16, "f16": sk.F16}


def parts(M, N, b, y):
    """Parts of the product of encoded rows: its workspace is their sums, rows padded to 4 outputs."""
    n = sk.sketch_int8_workspace_bytes(sk.Int8Params(M, N, 1), b, sk.INT8_ROWS, OUT[y])
    return n // ((M + 3) // 4 * 4 * b * 4)


@pytest.mark.parametrize("tile", PARTS)
def test_the_list_is_in_parts(tile):
    """For 16-bit outputs or for float32 (which decides between neighbouring tiles)."""
    found = [max(parts(*c, y) for y in DT) for c in PARTS[tile]]
    assert min(found) >= 2 and len(set(found)) >= 4, found


@pytest.mark.gpu
@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,b", LIST)
def test_products_in_parts(M, N, b, y):
    w, x = tables((M, N), M), tables((b, N), b)
    guard = 3.25 if y != "f32" else float(np.float32(3.3))
    out = torch.full((b * M + 64,), guard, dtype=DT[y], device=dev())
    n = sk.sketch_int8_workspace_bytes(w.params, b, sk.INT8_ROWS, OUT[y])
    ws = torch.full((n + 256,), 85, dtype=torch.uint8, device=dev())
    for _ in range(2):                        # the second on what the first left
        Y = out[:b * M].view(b, M).fill_(7.0)
        sk.int8_matmul(w, x, out=Y, workspace=ws)
        assert torch.equal(Y, product(x.codes(), x.scales(), w.codes(), w.scales(), DT[y]))
    assert (out[b * M:] == guard).all() and (ws[n:] == 85).all()
