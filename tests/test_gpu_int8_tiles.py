"""8-bit integer products at sizes that reach every kernel and tile, odd in every
direction, against float64 products of the codes (exact) on the GPU, bit for bit."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from int8_util import DT, ragged

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu


def tables(shape, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    codes = torch.randint(-127, 128, shape, generator=g, device=dev(), dtype=torch.int8)
    return sk.int8_tables(codes, torch.rand(shape[:-1], generator=g, device=dev()) * 0.01 + 1e-4)


def product(qx, sx, qw, sw, dtype):
    total = torch.matmul(qx.double(), qw.double().t().contiguous())
    return (total.float() * sx[:, None] * sw).to(dtype)


# M, N, rows: the smallest products found for each kind of tile and number of parts, for float32 or for 16 bits
DENSE = [(67, 74, 18), (71, 72, 39), (87, 3528, 17), (65, 2811, 37), (75, 2618, 44), (163, 64, 1814), (7493, 72, 33),
         (97, 5361, 302), (103, 4153, 275), (17435, 440, 68), (1617, 5680, 74), (1741, 4686, 80), (2273, 923, 907),
         (4759, 673, 391), (5873, 65, 1270), (8387, 68, 1275), (9269, 412, 1463), (19957, 143, 1378), (18993, 199, 1524), (13811, 129, 2035),
         (15183, 129, 1024), (12957, 106, 1275), (2304, 4096, 2048),
         (4096, 1024, 1537), (5000, 300, 2111)]


@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,b", DENSE)
def test_tiles(M, N, b, y):
    w, x = tables((M, N), M), tables((b, N), b)
    guard = 3.25 if y != "f32" else float(np.float32(3.3))
    out = torch.full((b * M + 64,), guard, dtype=DT[y], device=dev())
    Y = out[:b * M].view(b, M)
    sk.int8_matmul(w, x, out=Y)
    assert torch.equal(Y, product(x.codes(), x.scales(), w.codes(), w.scales(), DT[y]))
    assert (out[b * M:] == guard).all()


# experts, M, N, terms
GROUPS = [(3, 79, 130, 4), (8, 507, 589, 33), (20, 299, 565, 65), (3, 75, 70, 4), (8, 99, 71, 904), (3, 111, 72, 1008),
          (70, 983, 770, 256), (20, 4447, 779, 31), (8, 3261, 264, 2012), (8, 2657, 139, 3474), (20, 3015, 1610, 1461),
          (20, 3003, 646, 2372), (130, 515, 300, 2000), (4, 2048, 1024, 3000), (512, 33, 150, 9000), (1, 2600, 700, 1800)]


@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("E,M,N,terms", GROUPS)
def test_grouped_tiles(E, M, N, terms, gather, y):
    """Uneven groups, some of them empty, rows behind the last term, and rows of X in any order."""
    w, x = tables((E, M, N), M), tables((terms if not gather else terms // 3 + 1, N), terms)
    g = np.random.default_rng(terms)
    counts = ragged(E, terms - min(terms // 10, 40), terms + E, 0.2)
    rows = torch.from_numpy(g.integers(0, x.M, terms)).to(dev()) if gather else None
    out = torch.full((terms, M), 7.0, dtype=DT[y], device=dev())
    sk.int8_matmul_group(w, x, torch.tensor(counts, device=dev()), rows=rows, out=out)
    at = 0
    for e, n in enumerate(counts):
        if n:
            r = rows[at:at + n] if gather else torch.arange(at, at + n, device=dev())
            want = product(x.codes()[r], x.scales()[r], w.codes()[e], w.scales()[e], DT[y])
            assert torch.equal(out[at:at + n], want), e
            at += n
    assert (out[at:] == 7.0).all()


def test_every_width_of_a_last_tile():
    """Outputs and rows that end anywhere in a tile."""
    N = 256
    w, x = tables((300, N), 1), tables((300, N), 2)
    full = product(x.codes(), x.scales(), w.codes(), w.scales(), torch.bfloat16)
    for M in list(range(250, 300, 7)) + [257, 271, 289]:
        part = sk.int8_tables(w.codes()[:M].contiguous(), w.scales()[:M].contiguous())
        for b in (17, 63, 65, 127, 129, 255, 257, 300):
            rows = sk.int8_tables(x.codes()[:b].contiguous(), x.scales()[:b].contiguous())
            assert torch.equal(sk.int8_matmul(part, rows, dtype=torch.bfloat16), full[:b, :M]), (M, b)
