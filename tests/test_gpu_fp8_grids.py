"""Sizes whose workgroups are more than one dimension of a grid holds (2^32 - 1
threads), within the documented limits."""
import pytest
import torch

from gpu_util import dev

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

M = 1 << 24                  # SKETCH_FP8_MAX_M


def powers(count, dtype):
    """[count, M, 1]: 2^-3 .. 2^3, whose codes are 2^8 with a scale of their own."""
    return torch.exp2((torch.arange(count * M, device=dev()) % 7 - 3).to(dtype)).view(count, M, 1)


def test_rows_of_a_stack():
    W = powers(4, torch.float32)
    t = sk.fp8_encode(W, block_rows=1)
    assert (t.codes().view(torch.uint8) == 0x78).all()          # 256 = 2^8
    assert torch.equal(torch.exp2(t.scales().float() - 127) * 256, W)


def test_weights_of_a_stack():
    count = 33
    W = torch.zeros((count, M, 1), dtype=torch.bfloat16, device=dev())
    W[:, ::128] = powers(count, torch.float32)[:, ::128].to(torch.bfloat16)
    t = sk.fp8_encode(W, check=False)
    assert torch.equal(torch.exp2(t.scales().float() - 127) * 256, W[:, ::128].float())
    codes = t.codes().view(torch.uint8)
    assert (codes[:, ::128] == 0x78).all() and not codes[:, 1::128].any() and not codes[-1, 127::128].any()


def test_a_product_of_as_many_rows():
    N = 1537                     # 13 blocks, scales padded to 16
    w = torch.zeros((3, N), device=dev())
    w[0, 0], w[1, N - 1], w[2] = 2.0, 4.0, 1.0
    t = sk.fp8_encode(w)
    X = torch.ones((M, N), dtype=torch.bfloat16, device=dev())
    X[-1] = 2.0
    X[M // 2, N - 1] = 0.0
    want = torch.tensor([2.0, 4.0, 1537.0], device=dev()).repeat(M, 1)
    want[-1] *= 2
    want[M // 2] = torch.tensor([2.0, 0.0, 1536.0])
    assert torch.equal(sk.fp8_matmul(t, X), want)
