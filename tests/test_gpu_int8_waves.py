"""The row encoders of 8-bit integers on batches in which each row has a wave of
its own (rows of up to 2048 columns, from four for each compute unit on), against
the plain forms.  Odd numbers of rows leave the last workgroup short."""
import numpy as np
import pytest
import torch

import int8_util as u
from gpu_util import dev
from int8_util import DT, randn
from test_gpu_int8 import check_encode, check_swiglu

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

WIDTHS = [1, 7, 70, 128, 513, 1000, 1535, 2047, 2048]


def enough(more=1):
    dev()
    return 4 * torch.cuda.get_device_properties(0).multi_processor_count + more


def batch(rows, N, seed, dt):
    """`rows` spread over an ordinary batch, its first and last row among them; (the batch, where they are)."""
    M = enough()
    assert rows.shape[1] == N and rows.shape[0] <= M
    x = randn((M, N), seed, 1.0, dt)
    at = torch.linspace(0, M - 1, rows.shape[0]).long()
    x[at] = rows.to(DT[dt])
    return x, at


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_encode(N, dt):
    for more in (0, 1, 3):
        x = randn((enough(more), N), N + more, 0.3, dt)
        x[:, ::7] *= 30
        check_encode(x)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [381, 2048])
def test_encode_middles(N, dt):
    """Exact middles of two integers and their neighbours."""
    rows = []
    for amax in (127.0, 254.0, 1.984375, 1.0, 3.25, 1.9921875):
        mid = torch.tensor([(k + 0.5) / 127 * amax for k in range(127)], dtype=torch.float64).to(DT[dt])
        bits = mid.view(torch.int16 if dt != "f32" else torch.int32)
        near = torch.cat([(bits + d).view(DT[dt]) for d in (-1, 0, 1)])
        for sign in (1, -1):
            row = (near * sign).repeat(-(-N // 381))[:N].clone()
            row[N - 1] = amax
            rows.append(row)
    rows = torch.stack(rows)
    for e in (-20, 0) + ((-120, 100) if dt != "f16" else ()):
        check_encode(batch((rows.double() * 2.0 ** e).to(DT[dt]), N, 1, dt)[0])


@pytest.mark.parametrize("N", [70, 1000, 2048])
def test_encode_special_values(N):
    rows = torch.stack([torch.zeros(N), torch.full((N,), -0.0), torch.full((N,), 3.4e38), torch.full((N,), 2.0 ** -149),
                        torch.linspace(-1, 1, N) * 2.0 ** -126, torch.linspace(-1, 1, N) * 2.0 ** -100,
                        torch.linspace(-1, 1, N) * 3.4e38, torch.arange(N) * 2.0 ** -149])
    check_encode(batch(rows, N, 1, "f32")[0])
    rows[:, 0] = rows[:, 0].clamp(-3e38, 3e38)
    check_encode(batch(rows.clamp(-3e38, 3e38), N, 1, "bf16")[0])
    rows = torch.stack([torch.arange(N) * 2.0 ** -24, torch.full((N,), 65504.0), torch.linspace(-1, 1, N) * 2.0 ** -14])
    check_encode(batch(rows, N, 1, "f16")[0])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [3, 513, 2048])
def test_encode_non_finite_rows(N, dt):
    x = randn((enough(), N), 3, dt=dt)
    at = {0: "nan", 5: "inf", 6: "-inf", x.shape[0] - 1: "nan"}
    for i, (row, v) in enumerate(at.items()):
        x[row, (N - 1) * i // 3] = float(v)
    t = check_encode(x)
    assert torch.isnan(t.scales()).nonzero().flatten().tolist() == sorted(at)
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    sk.int8_encode(x.to(dev()), check=False, status=flags)
    assert int(flags) == sk.FLAG_WEIGHT_RANGE
    with pytest.raises(sk.SketchError):
        sk.int8_encode(x.to(dev()))
    flags.zero_()
    keep = [i for i in range(x.shape[0]) if i not in at] + [1, 2, 3, 4]
    sk.int8_encode(x[keep].to(dev()), check=False, status=flags)
    assert int(flags) == 0


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [70, 1000])
def test_encode_stacks_and_strides(N, dt):
    """Matrices that end inside a workgroup's four rows; rows with a stride, and not aligned to 16 bytes."""
    count = 7
    M = enough() // count + 1
    M += M % 2 == 0
    wide = randn((count, M, N + 30), 5, 1.0, dt).to(dev())
    for v in (wide[:, :, :N].contiguous(), wide[:, :, 3:3 + N]):
        t = sk.int8_encode(v)
        for i in range(count):
            q, s = u.encode(u.to64(v[i]))
            got, gs = u.table(t)
            assert np.array_equal(got[i], q) and np.array_equal(gs[i], s), i
        codes = t.buf.cpu().view(count, -1)[:, :M * t.layout.ld].reshape(count, M, t.layout.ld)
        assert not codes[:, :, N:].any()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_swiglu(N, dt):
    x = randn((enough(), 2 * N), N, 2.0, dt).to(dev())
    g, up = x[:, :N], x[:, N:]
    check_swiglu(g, up, sk.int8_swiglu(g, up))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [33, 600, 1100, 2048])
def test_swiglu_extremes(N, dt):
    """Far gates of both signs, values that only float64 holds on the way, rows of
    zeros, tiny rows, rows past float32's range, NaN and infinities, one row to a
    wave beside ordinary ones."""
    g, up = randn((14, N), 1, 1.0), randn((14, N), 2, 1.0)
    g[0], up[1] = 0.0, 0.0
    g[2] = -100.0
    g[3, N // 2], up[3, N // 2] = -89.0, 1e38
    g[4, N - 1], up[4, N - 1] = 1e30, 1e30
    g[5] *= 1e-25
    up[6] *= 1e-38
    g[7, N // 3] = float("nan")
    up[8, N - 2] = float("inf")
    g[9, 1] = float("-inf")
    g[10] = torch.linspace(-120, 120, N)
    g[11, 0], up[11, 0] = 1e19, 1e19
    g[12] = torch.linspace(-20, 0, N)
    g[13] *= 1e30
    G, at = batch(g, N, 3, dt)
    U, _ = batch(up, N, 4, dt)
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    t = sk.int8_swiglu(G.to(dev()), U.to(dev()), status=flags)
    check_swiglu(G, U, t)
    assert int(flags) == sk.FLAG_WEIGHT_RANGE
    bad = [4, 7, 8, 9]         # 1e19 * 1e19 is within float32
    assert torch.isnan(t.scales()).nonzero().flatten().tolist() == at[bad].tolist()
    G[at[bad]], U[at[bad]] = 1.0, 1.0
    flags.zero_()
    check_swiglu(G, U, sk.int8_swiglu(G.to(dev()), U.to(dev()), status=flags))
    assert int(flags) == 0
