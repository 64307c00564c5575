"""Tables of 8-bit integers that a caller fills in by hand, on the GPU."""
import pytest
import torch

from gpu_util import dev

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b", [1, 12, 40, 300])
def test_codes_filled_in_by_hand(b):
    """Tables made in memory that held something else give the products of the codes alone."""
    M, N = 70, 130
    g = torch.Generator(device=dev()).manual_seed(b)
    made = []
    for rows in (M, b):
        codes = torch.randint(-127, 128, (rows, N), generator=g, device=dev(), dtype=torch.int8)
        scales = torch.rand(rows, generator=g, device=dev())
        junk = torch.full((sk.sketch_int8_layout(sk.Int8Params(rows, N, 1)).bytes,), 85, dtype=torch.int8, device=dev())
        del junk                                  # its memory is the table's next
        t = sk.Int8Tables(rows, N, None, dev())
        t.codes().copy_(codes)
        t.scales().copy_(scales)
        made.append((t, codes, scales))
    (w, qw, sw), (x, qx, sx) = made
    total = torch.matmul(qx.double(), qw.double().t().contiguous()).float()
    assert torch.equal(sk.int8_matmul(w, x), total * sx[:, None] * sw)
