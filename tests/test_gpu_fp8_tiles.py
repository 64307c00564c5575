"""Products over the tiles and splits of K that their sizes choose."""
import pytest
import torch

from gpu_util import dev
from test_gpu_fp8 import small_ints

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("M,N,b", [
    (18432, 300, 17), (36900, 129, 33), (29000, 1100, 64),     # tall weights, few rows: small tiles
    (300, 2000, 65), (300, 2000, 129), (700, 700, 192),        # several tiles of 64 tokens
    (2100, 3000, 96), (2100, 3000, 191), (4099, 5003, 77),
    (18500, 300, 257), (9000, 1100, 384), (3000, 2100, 320),   # a last tile of 256 tokens mostly empty
    (17, 4000, 2500), (200, 1000, 5000), (500, 100, 2049)])
@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
def test_product(M, N, b, y):
    """Small integers: sums are exact on either kind of matrix core, so Y is the
    exact sum rounded once, by every tile and split."""
    w, x = small_ints((M, N), 1, 3), small_ints((b, N), 2, 4)
    t, xd = sk.fp8_encode(w.to(dev())), x.to(dev())
    want = (xd.double() @ w.to(dev()).double().t()).float().to(DT[y])
    Y = torch.full((b + 1, M), float("nan"), dtype=DT[y], device=dev())
    sk.fp8_matmul(t, xd, out=Y[:b])
    assert torch.equal(Y[:b], want) and torch.isnan(Y[b]).all()
    if y == "bf16":
        assert torch.equal(sk.fp8_matmul(t, xd, dtype=DT[y], float32_sums=True), want)


@pytest.mark.parametrize("M,N,b", [(5000, 2000, 77), (300, 3000, 150), (600, 1300, 520)])
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_repeats_are_identical(M, N, b, y):
    g = torch.Generator(device=dev()).manual_seed(3)
    t = sk.fp8_encode(torch.randn((M, N), generator=g, device=dev()))
    x = torch.randn((b, N), generator=g, device=dev())
    want = sk.fp8_matmul(t, x, dtype=DT[y])
    for _ in range(3):
        assert torch.equal(sk.fp8_matmul(t, x, dtype=DT[y]), want)


@pytest.mark.parametrize("b", [65535, 65536, 66000])
def test_parts_of_many_tokens(b):
    """Tokens up to and beyond a grid's second dimension, with few tiles."""
    w, x = small_ints((30, 1024), 1, 3), small_ints((b, 1024), 2, 4)
    t, xd = sk.fp8_encode(w.to(dev())), x.to(dev())
    want = (xd.double() @ w.to(dev()).double().t()).float()
    assert torch.equal(sk.fp8_matmul(t, xd), want)
