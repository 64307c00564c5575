"""The functions that carry the names of the C ABI, with every argument given by
hand, against the plain forms and the convenience layer."""
import numpy as np
import pytest
import torch

import int8_util as u
from gpu_util import dev
from int8_util import DT, randn

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

CODE = {"f32": sk.F32, "bf16": sk.BF16, "f16": sk.F16}


def words(n):
    return torch.zeros(n, dtype=torch.int32, device=dev())


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("other_stream", [False, True])
def test_encode(dt, other_stream):
    """Rows with a stride, in a stack, with the flags, on the current stream or on one that is given."""
    wide = randn((2, 21, 150), 4, 1.0, dt)
    wide[1, 3, 129] = float("inf")
    wide = wide.to(dev())
    W = wide[:, :, :130]
    p = sk.Int8Params(21, 130, 2)
    s = sk.sketch_int8_layout(p)
    buf, flags = torch.full((2 * s.bytes,), 85, dtype=torch.uint8, device=dev()), words(1)
    if other_stream:
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        sk.sketch_int8_encode(p, W, 150, buf, flags, stream.cuda_stream)
        stream.synchronize()
    else:
        sk.sketch_int8_encode(p, W, 150, buf, flags)
    t = sk.Int8Tables(21, 130, 2, dev(), buf)
    for i in range(2):
        q, sc = u.encode(u.to64(W[i]))
        got, gs = u.table(t)
        assert np.array_equal(got[i], q) and np.array_equal(gs[i], sc, equal_nan=True)
    assert int(flags) == sk.FLAG_WEIGHT_RANGE
    with pytest.raises(sk.SketchError) as e:
        sk.sketch_int8_encode(p, W, 129, buf)
    assert e.value.code == sk.EINVAL


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_swiglu(dt):
    x, up = randn((19, 400), 5, 1.5, dt).to(dev()), randn((19, 210), 6, 1.5, dt).to(dev())
    p = sk.Int8Params(19, 200, 1)
    t = sk.Int8Tables(19, 200, None, dev())
    flags = words(1)
    sk.sketch_int8_swiglu(p, x[:, 100:300], 400, up[:, :200], 210, t.buf, flags)
    want = sk.int8_swiglu(x[:, 100:300], up[:, :200])
    assert torch.equal(t.codes(), want.codes()) and torch.equal(t.scales(), want.scales()) and int(flags) == 0
    up[2, 3] = float("nan")
    sk.sketch_int8_swiglu(p, x[:, 100:300], 400, up[:, :200], 210, t.buf, flags)
    assert int(flags) == sk.FLAG_WEIGHT_RANGE and torch.isnan(t.scales()).nonzero().flatten().tolist() == [2]
    with pytest.raises(sk.SketchError):
        sk.sketch_int8_swiglu(p, x[:, 100:300], 400, up[:, :200], 199, t.buf)


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("b", [1, 9, 40, 200])
def test_matmul(x, y, b):
    w = sk.int8_encode(randn((130, 300), 2, 0.1).to(dev()))
    X = randn((b, 300), b, 1.0, x).to(dev())
    q, s = u.encode(u.to64(X))
    want = u.product(q, s, *u.table(w), y)
    p, Y = sk.Int8Params(130, 300, 1), torch.empty((b, 130), dtype=DT[y], device=dev())
    for rows, code in ((X, CODE[x]), (sk.int8_encode(X).buf, sk.INT8_ROWS)):
        n = sk.sketch_int8_workspace_bytes(p, b, code, CODE[y])
        assert n == (0 if (ws := sk.int8_workspace_for(w, b, code, CODE[y], dev())) is None else ws.numel())
        Y.fill_(7.0)
        sk.sketch_int8_matmul(p, w.buf, rows, code, b, Y, ws)
        u.same(Y, want)
        if n:
            with pytest.raises(sk.SketchError) as e:
                sk.sketch_int8_matmul(p, w.buf, rows, code, b, Y, ws[:n - 1])
            assert e.value.code == sk.ESMALL


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("T", [2, 30, 300])
@pytest.mark.parametrize("bits", [32, 64])
def test_matmul_group(x, y, T, bits):
    E, k = 5, 2
    w = sk.int8_encode(randn((E, 70, 300), 3, 0.1).to(dev()))
    X = randn((T, 300), T, 1.0, x).to(dev())
    g = np.random.default_rng(T)
    counts, rows = u.ragged(E, T * k - 1, T), g.integers(0, T, T * k)
    kind = torch.int32 if bits == 32 else torch.int64
    c, r = torch.tensor(counts, dtype=kind, device=dev()), torch.tensor(rows, dtype=kind, device=dev())
    q, s = u.encode(u.to64(X))
    start = randn((T * k, 70), 77, 1.0, y)
    want = u.group(q, s, rows, counts, *u.table(w), start)
    p = sk.Int8Params(70, 300, E)
    groups = sk.Int8Groups(T * k, c.data_ptr(), r.data_ptr(), bits, bits)
    for src, code in ((X, CODE[x]), (sk.int8_encode(X).buf, sk.INT8_ROWS)):
        n = sk.sketch_int8_group_workspace_bytes(p, T * k, T, code, CODE[y])
        ws = sk.int8_group_workspace_for(w, T * k, T, code, CODE[y], dev())
        assert n == (0 if ws is None else ws.numel())
        Y = start.to(dev())
        sk.sketch_int8_matmul_group(p, w.buf, src, code, T, groups, Y, ws)
        u.same(Y, want)
    with pytest.raises(sk.SketchError) as e:
        sk.sketch_int8_matmul_group(p, w.buf, X, CODE[x], 0, groups, Y, ws)
    assert e.value.code == sk.EINVAL
