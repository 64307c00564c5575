"""How the products of e4m3 codes are summed: in float32 for every type of Y and
number of rows, but for a bfloat16 Y of many rows that does not ask for it."""
import numpy as np
import pytest
import torch

import fp8_util as u
from gpu_util import dev

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# (M, N, b) of every kernel: a token, few tokens, few encoded rows, tiles of 64, 128 and 256 tokens, K split and not
SMALL = [(200, 500, 1), (200, 500, 4), (200, 500, 5), (200, 500, 16), (17000, 200, 9), (200, 500, 17), (200, 500, 64)]
LARGE = [(200, 500, 65), (700, 500, 300), (11000, 300, 250), (4300, 300, 2600), (4096, 256, 2560), (8200, 300, 1030)]


def cancelling(M, N, seed):
    """Weights whose groups of 8 hold a, -a and six values of up to 2^-17 of a:
    multiples of 2^-9 whose partial sums stay below 2^15 in any order, so that
    float32 holds every one of them."""
    g = np.random.default_rng(seed)
    n = u.blocks(N, 8)
    assert n * 448 < 2 ** 15
    w = g.integers(-7, 8, (M, n, 8)) * 2.0 ** -9
    a = g.integers(8, 15, (M, n)) * 32.0
    at = np.argsort(g.random((M, n, 8)), axis=2)[:, :, :2]
    np.put_along_axis(w, at[:, :, :1], a[:, :, None], axis=2)
    np.put_along_axis(w, at[:, :, 1:], -a[:, :, None], axis=2)
    w = w.reshape(M, n * 8)
    w[:, N // 8 * 8:] = 0
    w = w[:, :N]
    w[::128, ::128] = 448.0                      # the scale of every block is one
    w[::128, 1::128] = -448.0
    return torch.from_numpy(w.astype(np.float32))


def check_cancelling(M, N, b, y, **how):
    w = cancelling(M, N, M + N)
    x = torch.exp2((torch.arange(b) % 3).float())[:, None].expand(b, N).contiguous()
    t = sk.fp8_encode(w.to(dev()))
    assert np.array_equal(u.table_values(t)[:130], u.to64(w)[:130])
    want = torch.from_numpy(u.to64(x) @ u.to64(w).T).to(torch.float32).to(DT[y])
    assert torch.equal(sk.fp8_matmul(t, x.to(dev()), dtype=DT[y], **how).cpu(), want)


@pytest.mark.parametrize("M,N,b", SMALL + LARGE)
@pytest.mark.parametrize("y", ["f32", "f16"])
def test_float32_sums_of_products_that_cancel(M, N, b, y):
    check_cancelling(M, N, b, y)


@pytest.mark.parametrize("M,N,b", SMALL)
def test_few_rows_in_bfloat16_have_float32_sums(M, N, b):
    assert b <= sk.FP8_EXACT_BATCH
    check_cancelling(M, N, b, "bf16")


@pytest.mark.parametrize("M,N,b", LARGE)
def test_many_rows_in_bfloat16_have_float32_sums_when_asked(M, N, b):
    check_cancelling(M, N, b, "bf16", float32_sums=True)


def random_case(M, N, b, seed):
    """Normal weights, activations with a few large channels, and the product
    of the encoded values in float64 with the size of each output's products."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    w = torch.randn((M, N), generator=g, device=dev()).mul_(N ** -0.5).to(torch.bfloat16)
    x = torch.randn((b, N), generator=g, device=dev())
    x[:, ::50] *= 20
    t, r = sk.fp8_encode(w), sk.fp8_encode(x, block_rows=1)
    scale = lambda v, rows: torch.exp2(v.scales().double() - 127).repeat_interleave(rows, 0)[:v.M]
    val = lambda v, rows: v.codes().double() * scale(v, rows).repeat_interleave(128, 1)[:, :N]
    wv, xv = val(t, 128), val(r, 1)
    return t, r, xv @ wv.t(), ((xv ** 2) @ (wv ** 2).t()).sqrt()


@pytest.mark.parametrize("M,N,b", [(512, 8192, 1), (300, 9000, 12), (512, 8192, 64), (700, 5003, 77), (4096, 8192, 1100)])
@pytest.mark.parametrize("y", ["bf16", "f16"])
def test_float32_sums_in_16_bits(M, N, b, y):
    """Half a step of Y and a float32 sum's error, nothing else: n additions,
    each off by 2^-24 of a partial sum, walk to sqrt(n) * 2^-24 of the products'
    size; six times that."""
    t, r, ref, size = random_case(M, N, b, 1)
    Y = sk.fp8_matmul(t, r, dtype=DT[y], float32_sums=True).double()
    tol = 6 * N ** 0.5 * u.EPS32 * size
    # half a step of the value next to the border, and half of a binary16 subnormal's
    step = (ref.abs() + tol) * torch.finfo(DT[y]).eps / 2 + (2.0 ** -25 if y == "f16" else 0)
    assert ((Y - ref).abs() <= tol + step).all()


@pytest.mark.parametrize("M,N,b", [(4096, 8192, 1100), (1000, 16384, 200), (700, 5003, 77)])
def test_sums_on_the_e4m3_matrix_cores(M, N, b):
    """Many rows in bfloat16.  The sums are held to an error of rms 1e-4 of the
    products' size (twice what such data measured, 5e-5), seen through the
    rounding: an error d moves an output to the next bfloat16 value, a step s
    away, in a share d / s of the cases, so that the mean square of what is
    moved is at most the mean of d * s, with s <= 2^-7 * |y|; by Cauchy's
    inequality rms(d) * 2^-7 * rms(y).  And they have no bias beyond that: the
    mean of all errors, against six sigmas of the mean of the roundings."""
    t, r, ref, size = random_case(M, N, b, 2)
    fast = sk.fp8_matmul(t, r, dtype=torch.bfloat16).double()
    exact = sk.fp8_matmul(t, r, dtype=torch.bfloat16, float32_sums=True).double()
    d, rms = 1e-4 * size.square().mean().sqrt(), ref.square().mean().sqrt()
    assert (fast - exact).square().mean() <= d * 2.0 ** -7 * rms
    rounding = 2.0 ** -8 * rms / ref.numel() ** 0.5
    assert (fast - ref).mean().abs() <= d + 6 * rounding
    assert ((fast - ref) * ref.sign()).mean().abs() <= d + 6 * rounding


def test_a_workspace_for_float32_sums():
    M, N, b = 700, 2000, 300
    t = sk.fp8_encode(cancelling(M, 400, 1).repeat(1, 5).to(dev()))
    x = torch.ones(b, N, device=dev())
    ws = sk.fp8_workspace_for(t, b, sk.F32, sk.BF16 | sk.FP8_F32_SUMS, dev())
    Y = sk.fp8_matmul(t, x, dtype=torch.bfloat16, workspace=ws, float32_sums=True)
    assert torch.equal(Y, sk.fp8_matmul(t, x, dtype=torch.bfloat16, float32_sums=True))
    low = torch.empty_like(Y)
    sk.sketch_fp8_matmul(t.params, t.buf, x, sk.F32, b, low, ws, float32_sums=True)
    assert torch.equal(Y, low)
    # the other types have float32 sums in any case
    assert torch.equal(sk.fp8_matmul(t, x, float32_sums=True), sk.fp8_matmul(t, x))
