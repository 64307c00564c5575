"""Grouped products of 8-bit integers whose terms take rows in order beyond 4 GiB."""
import pytest
import torch

from gpu_util import dev

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_in_order_beyond_4_gib(dtype):
    """Without `rows` each tile counts from its own first term, so a batch of any
    size takes the tiles that its shape asks for: the bits are the codes' own."""
    R, N, M = 40000, 131071, 300
    g = torch.Generator(device=dev()).manual_seed(3)
    x = sk.Int8Tables(R, N, None, dev())
    for at in range(0, R, 4000):
        x.codes()[at:at + 4000] = torch.randint(-127, 128, (4000, N), generator=g, device=dev(), dtype=torch.int8)
    x.scales().copy_(torch.rand(R, generator=g, device=dev()) * 0.01)
    w = sk.int8_tables(torch.randint(-127, 128, (2, M, N), generator=g, device=dev(), dtype=torch.int8),
                       torch.rand(2, M, generator=g, device=dev()) * 0.01)
    for first in (5, 20001, R - 100):
        counts = torch.tensor([first, R - 50 - first], device=dev())
        out = torch.full((R, M), 7.0, dtype=dtype, device=dev())
        sk.int8_matmul_group(w, x, counts, out=out)
        some = torch.tensor([0, 1, 4, 5, 255, 256, 20000, 20001, 32766, 32767, 32768, 32769, R - 101, R - 100, R - 51], device=dev())
        total = torch.stack([torch.matmul(x.codes()[some].double(), c.double().t().contiguous()).float() for c in w.codes()])
        of = (some >= first).long()
        want = total[of, torch.arange(len(some), device=dev())] * x.scales()[some][:, None] * w.scales()[of]
        assert torch.equal(out[some], want.to(dtype)), first
        assert (out[R - 50:] == 7.0).all()
