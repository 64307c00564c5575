"""8-bit integer linears on the GPU against the plain forms: the encoder and
the product bit for bit (the sums are exact, so every variant of the kernels has
the same bits), SwiGLU's codes wherever extended precision tells the integer."""
import numpy as np
import pytest
import torch

import int8_util as u
from gpu_util import dev
from int8_util import DT, randn

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# encoder
# --------------------------------------------------------------------------

def check_encode(x, t=None):
    t = sk.int8_encode(x.to(dev()), check=False) if t is None else t
    q, s = u.encode(u.to64(x))
    got, gs = u.table(t)
    assert np.array_equal(gs, s, equal_nan=True)
    assert np.array_equal(got, q)
    codes = t.buf.cpu().numpy()[:t.M * t.layout.ld].reshape(t.M, t.layout.ld)
    assert not codes[:, t.N:].any()
    return t


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 128), (5, 127), (16, 129), (127, 256), (129, 1000), (3, 2048), (5, 2049),
                                 (3, 8192), (2, 8193), (2, 20001), (1, 131071), (1000, 70)])
def test_encode_bit_exact(M, N, dt):
    x = randn((M, N), M * 1000 + N, 0.3, dt)
    x[:, ::7] *= 30
    check_encode(x)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_encode_middles(dt):
    """Exact middles of two integers and their neighbours, at every scale of the type."""
    info = torch.finfo(DT[dt])
    rows = []
    for amax in (127.0, 254.0, 1.984375, 1.0, 3.25, 1.9921875):
        mid = torch.tensor([(k + 0.5) / 127 * amax for k in range(127)], dtype=torch.float64)
        v = mid.to(DT[dt])
        bits = v.view(torch.int16 if dt != "f32" else torch.int32)
        near = [(bits + d).view(DT[dt]) for d in (-1, 0, 1)]
        rows.append(torch.cat([torch.tensor([amax], dtype=DT[dt]), *near, -near[1]]))
    x = torch.stack(rows)
    for e in (-20, -2, 0, 6) + ((-120, 100) if dt != "f16" else ()):
        y = (x.to(torch.float64) * 2.0 ** e).to(DT[dt])
        assert torch.isfinite(y).all() and (y.abs().amax(1) <= info.max).all()
        check_encode(y)


def test_encode_special_values():
    """Rows of zeros, of signed zeros, subnormal, tiny and huge ones."""
    g = np.random.default_rng(5)
    rows = [torch.zeros(256), torch.full((256,), -0.0), torch.full((256,), 3.4e38), torch.full((256,), 2.0 ** -149),
            torch.linspace(-1, 1, 256) * 2.0 ** -126, torch.linspace(-1, 1, 256) * 2.0 ** -100,
            torch.linspace(-1, 1, 256) * 2.0 ** -121, torch.linspace(-1, 1, 256) * 3.4e38,
            torch.from_numpy(np.exp2(g.uniform(-140, 8, 256)).astype(np.float32)),
            torch.arange(256) * 2.0 ** -149]
    x = torch.stack(rows).to(torch.float32)
    check_encode(x)
    check_encode(x.to(torch.bfloat16).where(torch.isfinite(x.to(torch.bfloat16)), torch.tensor(3e38, dtype=torch.bfloat16)))
    h = torch.stack([torch.arange(256) * 2.0 ** -24, torch.full((256,), 65504.0), torch.linspace(-1, 1, 256) * 2.0 ** -14])
    check_encode(h.to(torch.float16))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [300, 3000])
def test_encode_non_finite_rows(N, dt):
    x = randn((9, N), 3, dt=dt)
    x[2, N - 1], x[4, 0], x[7, 5] = float("nan"), float("inf"), float("-inf")
    t = check_encode(x)
    assert int(torch.isnan(t.scales()).sum()) == 3
    with pytest.raises(sk.SketchError) as e:
        sk.int8_encode(x.to(dev()))
    assert e.value.code == sk.ERANGE
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    sk.int8_encode(x.to(dev()), check=False, status=flags)
    assert int(flags) == sk.FLAG_WEIGHT_RANGE
    flags.zero_()
    sk.int8_encode(x[:2].to(dev()), check=False, status=flags)
    assert int(flags) == 0


def test_encode_strides_and_stacks():
    x = randn((40, 700), 9, dt="bf16").to(dev())
    for v in (x[:, 3:600], x[::3, 1:130], x.t(), x[5:6, 2:4], x[:, :1], x[::2].t()):
        check_encode(v.cpu(), sk.int8_encode(v))
    y = randn((4, 30, 200), 10).to(dev())
    for v in (y, y[:, :, 5:150], y[:, 2:9], y[::2], y.transpose(0, 1), y[1:2, :, 7:]):
        t = sk.int8_encode(v)
        for i in range(v.shape[0]):
            q, s = u.encode(u.to64(v[i]))
            got, gs = u.table(t)
            assert np.array_equal(got[i], q) and np.array_equal(gs[i], s)
    assert sk.int8_encode(torch.zeros(0, 5, device=dev())).shape == (0, 5)


def test_tables_from_elsewhere():
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(-128, 128, (3, 20, 77), generator=g, dtype=torch.int8)
    scales = torch.rand(3, 20, generator=g)
    t = sk.int8_tables(codes.to(dev()), scales.to(dev()))
    got, gs = u.table(t)
    assert np.array_equal(got, codes.numpy()) and np.array_equal(gs, scales.numpy())
    assert int(t.codes().storage_offset()) == 0


# --------------------------------------------------------------------------
# SwiGLU and encoder
# --------------------------------------------------------------------------

def check_swiglu(g, up, t):
    """Codes as extended precision has them wherever the quotient is 1e-9 or more from a middle (the kernel's float64
    values are 1e-14 off at most); the scale within one rounding of float64 and one of float32."""
    h = u.swiglu(u.to64(g), u.to64(up))
    got, gs = u.table(t)
    with np.errstate(all="ignore"):
        big = np.abs(h).max(axis=1)
        bad = ~(big <= np.finfo(np.float32).max)
        want = np.where(bad, np.nan, (big / 127).astype(np.float64))
        assert np.array_equal(np.isnan(gs), bad)
        ok = ~bad
        assert (np.abs(gs[ok] - want[ok]) <= want[ok] * 2.0 ** -23 + 2.0 ** -149).all()
        q = np.where(bad[:, None] | (big == 0)[:, None], 0, 127 * h / np.where(big > 0, big, 1)[:, None])
    clear = np.abs(np.abs(q - np.floor(q)) - 0.5) > 1e-9
    assert clear.mean() > 0.99
    assert np.array_equal(got[clear], np.rint(q[clear]).astype(np.int64))
    assert (np.abs(got - q) <= 0.5 + 1e-9).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 1), (7, 1408), (33, 129), (5, 2048), (3, 2049), (64, 5000), (2, 11008), (1, 70000), (1100, 131)])
def test_swiglu(M, N, dt):
    x = randn((M, 2 * N), M + N, 2.0, dt).to(dev())
    g, up = x[:, :N], x[:, N:]
    check_swiglu(g, up, sk.int8_swiglu(g, up))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_swiglu_extremes(dt):
    """Far gates of both signs, values that only float64 holds on the way, rows
    of zeros, tiny rows, rows past float32's range, NaN and infinities."""
    n = 300
    g, up = randn((14, n), 1, 1.0).clone(), randn((14, n), 2, 1.0).clone()
    g[0], up[1] = 0.0, 0.0
    g[2] = -100.0
    g[3, 5], up[3, 5] = -89.0, 1e38
    g[4, 7], up[4, 7] = 1e30, 1e30
    g[5] *= 1e-25
    up[6] *= 1e-38
    g[7, 3] = float("nan")
    up[8, 4] = float("inf")
    g[9, 1] = float("-inf")
    g[10] = torch.linspace(-120, 120, n)
    g[11, 0], up[11, 0] = 1e19, 1e19
    g[12] = torch.linspace(-20, 0, n)
    g[13] *= 1e30
    g, up = g.to(DT[dt]).to(dev()), up.to(DT[dt]).to(dev())
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    t = sk.int8_swiglu(g, up, status=flags)
    check_swiglu(g, up, t)
    assert int(flags) == sk.FLAG_WEIGHT_RANGE
    flags.zero_()
    keep = [0, 1, 2, 3, 5, 6, 10, 11, 12, 13]
    check_swiglu(g[keep], up[keep], sk.int8_swiglu(g[keep], up[keep], status=flags))
    assert int(flags) == 0


def test_swiglu_strides():
    x = randn((20, 1000), 4, 1.5, "bf16").to(dev())
    y = randn((20, 400), 5, 1.5, "bf16").to(dev())
    for g, up in ((x[:, 3:400], x[:, 500:897]), (x[:, 1:401], y), (y[::3], x[::3, 7:407]), (y.t(), x[:, :400].t())):
        check_swiglu(g, up, sk.int8_swiglu(g, up))
    with pytest.raises(ValueError):
        sk.int8_swiglu(y, x)
    with pytest.raises(ValueError):
        sk.int8_swiglu(y, y.float())
    assert sk.int8_swiglu(y[:0], y[:0]).shape == (0, 400)


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------

def weight(M, N, seed):
    w = randn((M, N), seed, 0.05)
    w[::5] *= 7
    return sk.int8_encode(w.to(dev()))


def check_product(w, X, y, **more):
    q, s = u.encode(u.to64(X))
    want = u.product(q, s, *u.table(w), y)
    got = sk.int8_matmul(w, X, dtype=DT[y], **more)
    u.same(got, want)
    rows = sk.int8_encode(X, check=False)
    u.same(sk.int8_matmul(w, rows, dtype=DT[y]), want)
    return got


BATCHES = [1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 100, 127, 128, 129, 200, 256, 257, 400, 513]


@pytest.mark.parametrize("b", BATCHES)
@pytest.mark.parametrize("M,N", [(1, 1), (33, 130), (256, 512), (300, 1000), (515, 2050)])
def test_product(M, N, b):
    w = weight(M, N, M + N)
    x, y = [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")][(M + b) % 4]
    check_product(w, randn((b, N), b, 1.0, x).to(dev()), y)


@pytest.mark.parametrize("x", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("b", [1, 4, 7, 20, 70, 300])
def test_product_types(x, y, b):
    check_product(weight(130, 400, 3), randn((b, 400), b, 1.0, x).to(dev()), y)


@pytest.mark.parametrize("x", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(48, 1), (100, 2047), (33, 2049), (40, 5000), (40, 8200), (17, 16500), (16, 40000)])
@pytest.mark.parametrize("b", [1, 2, 3, 4, 7, 9, 16])
def test_product_of_raw_rows(M, N, b, x):
    """Rows that the product encodes itself: shorter and longer than its lanes keep, up to what LDS holds and beyond."""
    check_product(weight(M, N, M + N), randn((b, N), b, 1.0, x).to(dev()), "f32")


@pytest.mark.parametrize("M,N,b", [(4096, 4096, 1), (11008, 4096, 16), (4099, 5003, 77), (4096, 1024, 300), (1024, 8192, 700),
                                   (2000, 1408, 1000), (128, 20000, 40), (70001, 65, 3), (16, 131071, 18), (64, 131071, 1),
                                   (8192, 2048, 2049)])
def test_product_sizes(M, N, b):
    check_product(weight(M, N, M), randn((b, N), b, 1.0, "bf16").to(dev()), "bf16")


@pytest.mark.parametrize("b", [1, 16, 40, 130, 600])
def test_product_of_extreme_codes(b):
    """Sums at the ends of 32 bits: all codes -128 (as tables from elsewhere may
    have them) over the longest rows, one output with the other sign."""
    N = sk.INT8_MAX_N
    codes = torch.full((40, N), -128, dtype=torch.int8, device=dev())
    codes[7] = 127
    w = sk.int8_tables(codes, torch.full((40,), 0.5, device=dev()))
    x = sk.int8_tables(torch.full((b, N), -128, dtype=torch.int8, device=dev()), torch.full((b,), 3.0, device=dev()))
    got = sk.int8_matmul(w, x)
    want = torch.full((b, 40), float(np.float32(128 * 128 * N) * np.float32(3.0) * np.float32(0.5)))
    want[:, 7] = float(np.float32(-128 * 127 * N) * np.float32(3.0) * np.float32(0.5))
    u.same(got, want)


@pytest.mark.parametrize("b", [3, 12, 50, 200])
def test_product_non_finite_rows_and_channels(b):
    """NaN and infinities stay in their rows; a channel with the scale NaN in its column; overflow of binary16 to infinity."""
    w = weight(200, 300, 8)
    X = randn((b, 300), 5, 1.0, "bf16").to(dev())
    clean = sk.int8_matmul(w, X)
    X[1, 7], X[2, 0] = float("nan"), float("inf")
    Y = sk.int8_matmul(w, X)
    assert torch.isnan(Y[1:3]).all()
    keep = [i for i in range(b) if i not in (1, 2)]
    assert torch.equal(Y[keep], clean[keep])
    w.scales()[11] = float("nan")
    w.scales()[12] = 1e30
    Y = sk.int8_matmul(w, X, dtype=torch.float16)
    assert torch.isnan(Y[:, 11]).all() and torch.isinf(Y[keep][:, 12]).all()


def test_out_workspace_strides_vectors():
    w = weight(130, 384, 2)
    X = randn((50, 384), 6, 1.0, "bf16").to(dev())
    want = sk.int8_matmul(w, X, dtype=torch.bfloat16)
    out = torch.empty((50, 130), dtype=torch.bfloat16, device=dev())
    ws = sk.int8_workspace_for(w, 50, sk.BF16, sk.BF16, dev())
    assert sk.int8_matmul(w, X, out=out, workspace=ws) is out
    assert torch.equal(out, want)
    one = sk.int8_matmul(w, X[3], dtype=torch.bfloat16)
    assert one.shape == (130,) and torch.equal(one, want[3])
    big = torch.zeros((100, 800), dtype=torch.bfloat16, device=dev())
    big[::2, 3:387] = X
    assert torch.equal(sk.int8_matmul(w, big[::2, 3:387], dtype=torch.bfloat16), want)
    assert torch.equal(sk.int8_matmul(w, X.t().contiguous().t(), dtype=torch.bfloat16), want)
    assert sk.int8_matmul(w, X[:0]).shape == (0, 130)
    for bad in (torch.empty((50, 131), device=dev()), torch.empty((50, 260), device=dev())[:, ::2]):
        with pytest.raises(ValueError):
            sk.int8_matmul(w, X, out=bad)
    with pytest.raises(ValueError):
        sk.int8_matmul(w, X, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(sk.SketchError) as e:
        sk.int8_matmul(w, X, workspace=ws[:16])
    assert e.value.code == sk.ESMALL


@pytest.mark.parametrize("b", [1, 4, 5, 16, 17, 40, 200])
def test_out_may_be_x(b):
    w = weight(256, 256, 4)
    X = randn((b, 256), 6).to(dev())
    want = sk.int8_matmul(w, X)
    sk.int8_matmul(w, X, out=X)
    assert torch.equal(X, want)


@pytest.mark.parametrize("b", [1, 3, 12, 40, 150, 600])
def test_in_a_graph_with_new_inputs(b):
    w = weight(515, 1000, 1)
    X = randn((b, 1000), 0, 1.0, "bf16").to(dev())
    Y = torch.empty((b, 515), device=dev())
    ws = sk.int8_workspace_for(w, b, sk.BF16, sk.F32, dev())
    sk.int8_matmul(w, X, out=Y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sk.int8_matmul(w, X, out=Y, workspace=ws)
    for i in range(1, 4):
        X.copy_(randn((b, 1000), i, 1.0, "bf16"))
        want = sk.int8_matmul(w, X)
        Y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want), i


def test_on_another_stream_and_two_at_once():
    w = weight(1000, 2048, 1)
    Xs = [randn((b, 2048), b, 1.0, "bf16").to(dev()) for b in (60, 300)]
    want = [sk.int8_matmul(w, X) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = [[] for _ in Xs]
    for _ in range(3):
        for i, (s, X) in enumerate(zip(streams, Xs)):
            with torch.cuda.stream(s):
                got[i].append(sk.int8_matmul(w, X))
    torch.cuda.synchronize()
    for g, y in zip(got, want):
        assert all(torch.equal(v, y) for v in g)


def test_weight_beyond_4_gib():
    """Rows whose codes lie past 2^32 bytes."""
    M, N = 40000, 131071
    w = sk.Int8Tables(M, N, None, dev())
    g = torch.Generator(device=dev()).manual_seed(3)
    w.buf.zero_()
    at = [0, 1, 16383, 32767, 32768, 32769, M - 2, M - 1]
    codes = torch.randint(-127, 128, (len(at), N), generator=g, device=dev(), dtype=torch.int8)
    w.codes()[at] = codes
    w.scales()[at] = 1.0
    for b in (2, 30, 140):
        x = sk.int8_encode(randn((b, N), b, 1.0, "bf16").to(dev()))
        Y = sk.int8_matmul(w, x)
        q, s = u.table(x)
        want = u.product(q, s, codes.cpu().numpy().astype(np.int64), np.ones(len(at), np.float32), "f32")
        u.same(Y[:, at], want)
        Y[:, at] = 0
        assert not Y.any()
