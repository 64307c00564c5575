"""e4m3 linears on the GPU against the plain 64-bit forms: the encoder bit for
bit; the product bit for bit on inputs whose sums are exact in float32 in any
order, and within a derived tolerance on random ones."""
import numpy as np
import pytest
import torch

import fp8_util as u
from gpu_util import dev

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def randn(shape, seed, scale=1.0, dt="f32"):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(DT[dt])


# --------------------------------------------------------------------------
# encoder
# --------------------------------------------------------------------------

def check_encode(x, rows):
    t = sk.fp8_encode(x.to(dev()), block_rows=rows, check=False)
    want, byte = u.encode(u.to64(x), rows)
    got = u.e4m3_value(t.codes().view(torch.uint8).cpu().numpy())
    assert np.array_equal(t.scales().cpu().numpy(), byte)
    assert np.array_equal(got, want, equal_nan=True)
    # padding: columns N..ld and the scale bytes that round a row up are zero
    s, flat = t.layout, t.buf.cpu().numpy()
    codes = flat[:t.M * s.ld].reshape(t.M, s.ld)
    assert not codes[:, t.N:].any()
    sc = flat[s.scales_offset:s.scales_offset + s.row_blocks * s.lds].reshape(s.row_blocks, s.lds)
    assert not sc[:, s.col_blocks:].any()
    return t


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 128), (5, 127), (16, 129), (127, 256), (129, 1000), (300, 515),
                                 (256, 512)])
def test_encode_bit_exact(M, N, rows, dt):
    x = randn((M, N), M * 1000 + N, 0.3, dt)
    x[:, ::7] *= 30
    check_encode(x, rows)


@pytest.mark.parametrize("rows", [1, 128])
def test_encode_special_values(rows):
    """All-zero blocks, the edges of a scale, subnormal and huge magnitudes,
    signed zeros, ties between codes."""
    blocks = [torch.zeros(128), torch.full((128,), -0.0), torch.full((128,), 448.0),
              torch.full((128,), 448.0).nextafter(torch.tensor(1e9)), torch.full((128,), 3.0e38),
              torch.full((128,), 2.0 ** -149), torch.full((128,), 448 * 2.0 ** -130), torch.full((128,), 2.0 ** -133)]
    t = torch.linspace(-448, 448, 128)
    blocks += [t, t * 2.0 ** -20, torch.arange(128) * 0.0625 + 16, torch.arange(128) * 0.5 + 100]
    g = np.random.default_rng(5)
    blocks.append(torch.from_numpy(np.exp2(g.uniform(-140, 8, 128)).astype(np.float32)))
    check_encode(torch.cat(blocks)[None, :].to(torch.float32), rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_encode_non_finite_blocks(rows, bad):
    """A block with NaN or an infinity is NaN as a whole, the others are as
    without it, the flag is raised; the padding stays zero."""
    x = randn((130, 300), 3, dt="bf16")
    x[129, 299] = bad
    t = check_encode(x, rows)
    assert t.scales().cpu().numpy()[-1, -1] == 255
    assert int((t.scales() == 255).sum()) == 1
    with pytest.raises(sk.SketchError) as e:
        sk.fp8_encode(x.to(dev()), block_rows=rows)
    assert e.value.code == sk.ERANGE
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    sk.fp8_encode(x.to(dev()), block_rows=rows, check=False, status=flags)
    assert int(flags.item()) == sk.FLAG_WEIGHT_RANGE
    flags.zero_()
    sk.fp8_encode(x[:, :256].to(dev()), block_rows=rows, check=False, status=flags)
    assert int(flags.item()) == 0


def test_encode_stack_and_strided_inputs():
    x = randn((3, 140, 200), 9, dt="bf16")
    t = sk.fp8_encode(x.to(dev()))
    for i in range(3):
        one = check_encode(x[i], 128)
        assert torch.equal(one.codes().view(torch.uint8), t.codes()[i].view(torch.uint8))
        assert torch.equal(one.scales(), t.scales()[i])
    wide = x[0].to(dev())
    a, b = sk.fp8_encode(wide.t()), sk.fp8_encode(wide.t().contiguous())
    assert torch.equal(a.codes().view(torch.uint8), b.codes().view(torch.uint8))
    off = torch.cat([torch.zeros(1, dtype=torch.bfloat16, device=dev()), wide.flatten()])[1:].view(140, 200)
    assert off.data_ptr() % 16 != 0
    assert torch.equal(sk.fp8_encode(off).scales(), sk.fp8_encode(wide).scales())


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------

def small_ints(shape, seed, top, dt="f32"):
    """Integers of magnitude up to `top`, with `top` in every 128 columns."""
    g = np.random.default_rng(seed)
    x = g.integers(-top, top + 1, shape).astype(np.float32)
    x[..., ::128] = top
    return torch.from_numpy(x).to(DT[dt])


def exact_case(M, N, b, dt, seed=0):
    """Integer operands whose products' sums stay below 2^24 times the unit of
    the products, so float32 gives them exactly in any order; power-of-two
    factors of their own for every row and block tell scales apart."""
    g = np.random.default_rng(seed + 77)
    w = small_ints((M, N), seed, 3)
    x = small_ints((b, N), seed + 1, 4, dt)
    f = torch.from_numpy(np.exp2(g.integers(-3, 4, (u.blocks(M, 128),))).astype(np.float32))
    w = w * f.repeat_interleave(128)[:M, None]
    fx = torch.from_numpy(np.exp2(g.integers(-3, 4, (b,))).astype(np.float32))
    x = x * fx[:, None].to(x.dtype)
    # column block j is 2^(j % 3) as large in the weight
    fk = torch.exp2((torch.arange(u.blocks(N, 128)) % 3).float()).repeat_interleave(128)[:N]
    w = w * fk
    assert N * 12 * 4 < 2 ** 24
    return w, x


BATCHES = [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 257]
SHAPES = [(1, 1), (16, 128), (15, 127), (129, 257), (256, 512), (1000, 1111), (513, 2048)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("b", BATCHES)
def test_product_exact(M, N, b):
    w, x = exact_case(M, N, b, "bf16", M + N + b)
    assert np.array_equal(u.encoded(u.to64(w), 128), u.to64(w)) and np.array_equal(u.encoded(u.to64(x), 1), u.to64(x))
    t = sk.fp8_encode(w.to(dev()))
    Y = torch.full((b, M), float("nan"), device=dev())
    sk.fp8_matmul(t, x.to(dev()), out=Y)
    assert np.array_equal(u.to64(Y), u.to64(x) @ u.to64(w).T)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,b", [(300, 4001, 1), (300, 4001, 9), (2050, 640, 40), (700, 900, 300), (4096, 11008, 3),
                                   (384, 300, 2000), (130, 11008, 140), (2100, 2500, 1300),
                                   (4333, 4300, 13), (16400, 200, 16), (11008, 500, 480), (6000, 1000, 130), (8200, 1155, 1030), (4099, 1, 3001)])
def test_product_exact_larger(M, N, b, dt):
    w, x = exact_case(M, N, b, dt, 5)
    t = sk.fp8_encode(w.to(dev()))
    assert np.array_equal(u.to64(sk.fp8_matmul(t, x.to(dev()))), u.to64(x) @ u.to64(w).T)


@pytest.mark.parametrize("M,N,b", [(16, 128, 70), (700, 900, 1), (513, 1300, 65), (1000, 1111, 300), (2050, 640, 128),
                                   (4300, 300, 3000), (4097, 1, 3001), (5000, 1155, 2570), (130, 11008, 140), (11000, 900, 250), (6001, 1000, 129)])
@pytest.mark.parametrize("y", ["bf16", "f16"])
def test_product_in_16_bits(M, N, b, y):
    """Small integers: groups of 8 products, and all sums, are exact on either
    kind of matrix core, so Y is the exact sum rounded once."""
    w, x = small_ints((M, N), 1, 3), small_ints((b, N), 2, 4)
    t = sk.fp8_encode(w.to(dev()))
    want = torch.from_numpy(u.to64(x) @ u.to64(w).T).to(torch.float32).to(DT[y])
    out = torch.full((b, M), float("nan"), dtype=DT[y], device=dev())
    assert torch.equal(sk.fp8_matmul(t, x.to(dev()), out=out).cpu(), want)
    assert torch.equal(sk.fp8_matmul(t, x.to(dev()), dtype=DT[y]).cpu(), want)


@pytest.mark.parametrize("M,N,b", [(512, 4096, 1), (300, 1000, 16), (700, 5003, 77), (512, 2048, 300)])
def test_product_random(M, N, b):
    """Rounding of a float32 sum of n products: each addition is off by at most
    2^-24 of a partial sum, of size about sqrt(n) times a product's; n of them
    add up like a random walk to sqrt(n) * 2^-24 of the sum's own size.  Six
    times that, on the size sqrt(sum of squares) of each output.

    In 16 bits: half a step of Y, and the e4m3 matrix cores' 13 bits below the largest product p of 8 neighbours: 7 * 2^-13 * |p|."""
    w, x = randn((M, N), 1, 0.02, "bf16"), randn((b, N), 2, 1.0, "bf16")
    x[:, ::50] *= 20
    t = sk.fp8_encode(w.to(dev()))
    wv, xv = u.table_values(t), u.encoded(u.to64(x), 1)
    ref = xv @ wv.T
    tol = 6 * np.sqrt(N) * u.EPS32 * np.sqrt((xv ** 2) @ (wv ** 2).T)
    assert (np.abs(u.to64(sk.fp8_matmul(t, x.to(dev()))) - ref) <= tol).all()
    for y in ("bf16", "f16"):
        err = np.abs(u.to64(sk.fp8_matmul(t, x.to(dev()), dtype=DT[y])) - ref)
        step = np.abs(ref) * torch.finfo(DT[y]).eps / 2 + (2.0 ** -25 if y == "f16" else 0)
        groups = np.zeros_like(ref)
        n8 = N // 8 * 8
        for i in range(b):
            p = np.abs(xv[i, :n8].reshape(-1, 8)[None] * wv[:, :n8].reshape(M, -1, 8)).max(2).sum(1)
            groups[i] = 7 * 2.0 ** -13 * (p + (np.abs(xv[i, n8:] * wv[:, n8:]).max(1) if N > n8 else 0))
        assert (err <= tol + step * (1 + 2.0 ** -8) + groups).all(), y


@pytest.mark.parametrize("b", [1, 7, 16, 40, 200])
def test_encoded_rows_give_the_same_bits(b):
    w, x = randn((500, 1300), 3, 0.1), randn((b, 1300), 4, 2.0, "f16").to(dev())
    t = sk.fp8_encode(w.to(dev()))
    Y = sk.fp8_matmul(t, x)
    assert torch.equal(Y, sk.fp8_matmul(t, sk.fp8_encode(x, block_rows=1)))
    assert torch.equal(Y, sk.fp8_matmul(t, x))                                # and again


@pytest.mark.parametrize("M,N,b", [(100, 300, 3), (200, 700, 20), (200, 700, 150), (5000, 300, 2600)])
def test_non_finite_rows_and_weights_in_16_bits(M, N, b):
    """NaN in a row of X, or in a block of W, reaches its row (its outputs)
    and nothing else, on the e4m3 matrix cores too."""
    w, x = small_ints((M, N), 1, 3), small_ints((b, N), 2, 4)
    x[1, 5] = float("inf")
    t = sk.fp8_encode(w.to(dev()))
    with np.errstate(invalid="ignore"):
        want = torch.from_numpy(u.to64(x) @ u.to64(w).T).to(torch.bfloat16)
    Y = sk.fp8_matmul(t, x.to(dev()), dtype=torch.bfloat16).cpu()
    keep = torch.arange(b) != 1
    assert torch.isnan(Y[1].float()).all() and torch.equal(Y[keep], want[keep])
    w[M - 1, N - 1], x[1, 5] = float("nan"), 0.0
    t = sk.fp8_encode(w.to(dev()), check=False)
    Y = sk.fp8_matmul(t, x.to(dev()), dtype=torch.bfloat16).cpu()
    first = (M - 1) // 128 * 128
    want = torch.from_numpy(u.to64(x) @ u.to64(w[:first]).T).to(torch.bfloat16)
    assert torch.isnan(Y[:, first:].float()).all() and torch.equal(Y[:, :first], want)


@pytest.mark.parametrize("b", [1, 9, 40])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -108, 2.0 ** 100])
def test_far_scales(b, y, scale):
    """Weights far from one: sums stay exact (small integers times the scale)."""
    w, x = small_ints((130, 400), 1, 3), small_ints((b, 400), 2, 4)
    t = sk.fp8_encode((w * scale).to(dev()))
    want = torch.from_numpy(u.to64(x) @ u.to64(w).T * scale).to(torch.float32).to(DT[y])
    assert torch.equal(sk.fp8_matmul(t, x.to(dev()), dtype=DT[y]).cpu(), want)


@pytest.mark.parametrize("M,b,y", [(130, 1, "f32"), (130, 1, "bf16"), (130, 9, "f32"), (130, 9, "bf16"), (130, 40, "f32"),
                                   (130, 200, "bf16"), (5000, 2600, "bf16"), (5001, 2600, "f32")])
@pytest.mark.parametrize("byte,other", [(0, 217), (1, 187), (9, 150), (247, 60), (254, 50)])
def test_scale_bytes_at_their_ends(M, b, y, byte, other):
    """Tables from elsewhere with scales up to the ends of their range, on the
    weight and on the rows: even integers, so that at 2^-127 every element is
    at least 2^-126, and at 2^127 only ones; sums stay exact."""
    N = 300
    w, x = small_ints((M, N), 1, 3), small_ints((b, N), 2, 3)
    w, x = (w.clamp(-1, 1), x.clamp(-1, 1)) if byte == 254 else (w * 2, x * 2)
    codes = lambda a: a.to(dev()).to(torch.float8_e4m3fn)
    full = lambda rows, e: torch.full((rows, 3), e, dtype=torch.uint8, device=dev())
    for we, xe in ((byte, other), (other, byte)):
        t = sk.fp8_tables(codes(w), full(u.blocks(M, 128), we))
        r = sk.fp8_tables(codes(x), full(b, xe), block_rows=1)
        want = torch.from_numpy(u.to64(x) @ u.to64(w).T * 2.0 ** (we + xe - 254)).to(torch.float32).to(DT[y])
        assert torch.equal(sk.fp8_matmul(t, r, dtype=DT[y]).cpu(), want), (we, xe)


@pytest.mark.parametrize("M,b,y", [(300, 1, "f32"), (300, 3, "bf16"), (300, 9, "f32"), (300, 40, "f32"),
                                   (300, 200, "bf16"), (5000, 2600, "bf16"), (5001, 2600, "f32")])
@pytest.mark.parametrize("code", [0.0, 1.0, -448.0])
def test_a_nan_scale_is_nan_whatever_its_codes(M, b, y, code):
    """The scale byte 255 over ordinary codes, zeros among them, in a block of
    the weight and in a row's block: NaN for its outputs, its row, no others."""
    N = 300
    w, x = small_ints((M, N), 1, 3), small_ints((b, N), 2, 3)
    w[128:256, 256:] = code
    t, r = sk.fp8_encode(w.to(dev())), sk.fp8_encode(x.to(dev()), block_rows=1)
    t.scales()[1, 2] = 255
    Y = sk.fp8_matmul(t, r, dtype=DT[y]).cpu()
    keep = torch.ones(M, dtype=torch.bool)
    keep[128:256] = False
    want = torch.from_numpy(u.to64(x) @ u.to64(w).T).to(torch.float32).to(DT[y])
    assert torch.isnan(Y[:, ~keep]).all() and torch.equal(Y[:, keep], want[:, keep])
    x[b // 2, 128:256] = code
    r = sk.fp8_encode(x.to(dev()), block_rows=1)
    r.scales()[b // 2, 1] = 255
    Y = sk.fp8_matmul(t, r, dtype=DT[y]).cpu()
    rows = torch.arange(b) != b // 2
    assert torch.isnan(Y[b // 2]).all() and torch.equal(Y[rows][:, keep], want[rows][:, keep])


@pytest.mark.parametrize("b", [3, 20, 150])
def test_zero_rows_blocks_and_non_finite_rows(b):
    """Zero rows and zero blocks give zeros; NaN and infinities stay in their row."""
    w, x = exact_case(200, 700, b, "f32", 11)
    x[0] = 0
    w[:, 128:256] = 0
    x[1, 5], x[2, 699] = float("nan"), float("-inf")
    t = sk.fp8_encode(w.to(dev()))
    Y = u.to64(sk.fp8_matmul(t, x.to(dev())))
    ok = np.arange(b) % b > 2
    ok[0] = True
    assert np.isnan(Y[1]).all() and np.isnan(Y[2]).all()
    assert np.array_equal(Y[ok], u.to64(x)[ok] @ u.to64(w).T)


def test_tables_from_codes_and_scales():
    w = randn((2, 200, 300), 8, 0.1)
    t = sk.fp8_encode(w.to(dev()))
    s = t.scales().contiguous()
    r = sk.fp8_tables(t.codes(), s)
    r2 = sk.fp8_tables(t.codes().view(torch.uint8), s.view(torch.float8_e8m0fnu))
    assert torch.equal(r.buf, r2.buf) and torch.equal(r.scales(), t.scales())
    assert torch.equal(r.codes().view(torch.uint8), t.codes().view(torch.uint8))
    for c, e in ((t.codes(), s[:, :1]), (t.codes().view(torch.uint8).view(torch.float8_e5m2), s),
                 (t.codes(), s.float()), (t.codes().float(), s)):
        with pytest.raises(ValueError):
            sk.fp8_tables(c, e)


def test_rows_behind_the_output_are_left_alone():
    for b, M in ((3, 37), (16, 300), (70, 130)):
        w, x = exact_case(M, 256, b, "bf16", 3)
        t = sk.fp8_encode(w.to(dev()))
        big = torch.full((b + 40, M), 7.0, device=dev())
        sk.fp8_matmul(t, x.to(dev()), out=big[:b])
        assert (big[b:] == 7.0).all()
        assert np.array_equal(u.to64(big[:b]), u.to64(x) @ u.to64(w).T)


def test_other_stream_and_refused_outputs():
    w, x = exact_case(256, 512, 5, "bf16", 2)
    t, xd = sk.fp8_encode(w.to(dev())), x.to(dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Y = sk.fp8_matmul(t, xd)
    s.synchronize()
    assert np.array_equal(u.to64(Y), u.to64(x) @ u.to64(w).T)
    for out in (torch.empty(5, 255, device=dev()), torch.empty(5, 256, device=dev(), dtype=torch.float16),
                torch.empty(256, 5, device=dev()).t(), torch.empty(5, 256)):
        with pytest.raises(ValueError):
            sk.fp8_matmul(t, xd, out=out, dtype=torch.float32)
    with pytest.raises(TypeError):
        sk.fp8_matmul(t, xd, out=torch.empty(5, 256, device=dev(), dtype=torch.float64))
    with pytest.raises(ValueError):
        sk.fp8_matmul(t, x)                               # X on the host
    with pytest.raises(ValueError):
        sk.fp8_matmul(t, xd, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        sk.fp8_encode(w.to(dev()), check=False, status=torch.zeros(1, dtype=torch.int32))
    assert sk.fp8_matmul(t, xd[:0]).shape == (0, 256)
    assert np.array_equal(u.to64(sk.fp8_matmul(t, xd[2])), u.to64(x)[2] @ u.to64(w).T)


def test_offsets_beyond_32_bits():
    """A weight of more than 4 GiB of codes: its last block encoded, and read
    by every kind of product."""
    M, N = 70016, 65536
    g = torch.Generator(device=dev()).manual_seed(1)
    W = torch.zeros((M, N), dtype=torch.bfloat16, device=dev())
    W[-128:] = torch.randint(-3, 4, (128, N), generator=g, device=dev()).to(torch.bfloat16)
    W[-128:, ::128] = 3
    t = sk.fp8_encode(W, check=False)
    last = W[-128:].clone()
    del W
    one = sk.fp8_encode(last)
    assert torch.equal(t.codes()[-128:].view(torch.uint8), one.codes().view(torch.uint8))
    assert torch.equal(t.scales()[-1], one.scales()[0]) and not t.codes()[:-128].view(torch.uint8).any()
    for b, y in ((1, "f32"), (9, "bf16"), (33, "f32"), (200, "bf16")):
        x = torch.randint(-3, 4, (b, N), generator=g, device=dev()).to(torch.bfloat16)
        x[:, ::128] = 3
        want = (x.double() @ last.double().t()).float().to(DT[y])
        Y = sk.fp8_matmul(t, x, dtype=DT[y])
        assert torch.equal(Y[:, -128:], want) and not Y[:, :-128].any()


@pytest.mark.parametrize("b", [1, 16, 40, 300])
def test_captured_and_replayed(b):
    """The whole call in a graph, replayed on new inputs between eager calls."""
    M, N = 384, 1000
    w, _ = exact_case(M, N, b, "bf16", 4)
    t = sk.fp8_encode(w.to(dev()))
    xs = [exact_case(M, N, b, "bf16", 50 + i)[1].to(dev()) for i in range(3)]
    x, Y = xs[0].clone(), torch.empty(b, M, device=dev())
    ws = sk.fp8_workspace_for(t, b, sk.BF16, sk.F32, dev())
    sk.fp8_matmul(t, x, out=Y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.fp8_matmul(t, x, out=Y, workspace=ws)
    for xi in xs:
        x.copy_(xi)
        Y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        eager = sk.fp8_matmul(t, xi)
        assert torch.equal(Y, eager)
        assert np.array_equal(u.to64(Y), u.to64(xi) @ u.to64(w).T)


def test_many_rows_of_a_narrow_weight():
    """More tokens than a grid's second dimension holds, few outputs."""
    w, x = small_ints((40, 200), 1, 3), small_ints((70001, 200), 2, 4)
    t = sk.fp8_encode(w.to(dev()))
    want = torch.from_numpy(u.to64(x) @ u.to64(w).T).to(torch.float32)
    for y in ("f32", "bf16"):
        assert torch.equal(sk.fp8_matmul(t, x.to(dev()), dtype=DT[y]).cpu(), want.to(DT[y]))


def test_encoder_captured_and_replayed():
    """New weights and new rows at each replay, between eager calls."""
    ws = [randn((200, 300), 20 + i, 0.1).to(dev()) for i in range(3)]
    xs = [randn((9, 300), 30 + i, 1.0, "bf16").to(dev()) for i in range(3)]
    W, X, flags = ws[0].clone(), xs[0].clone(), torch.zeros(1, dtype=torch.int32, device=dev())

    def step():
        rows = sk.fp8_encode(X, block_rows=1, check=False)
        return sk.fp8_matmul(sk.fp8_encode(W, check=False, status=flags), rows)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = step()
    for w, x in zip(ws, xs):
        W.copy_(w), X.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, sk.fp8_matmul(sk.fp8_encode(w), x)) and int(flags.item()) == 0
    W[3, 4] = float("inf")
    g.replay()
    torch.cuda.synchronize()
    assert int(flags.item()) == sk.FLAG_WEIGHT_RANGE and torch.isnan(Y[:, :128]).all()
