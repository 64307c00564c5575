"""Buffers of one call of the 8-bit integer products that share memory are
refused before anything is enqueued (no GPU: a call that is not refused fails at
its launch, with another code)."""
import ctypes

import pytest

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

vp = ctypes.c_void_p
AT = 1 << 32               # buffers lie at multiples of this


def place(size, at):
    """Addresses apart, but for the buffers that `at` places on another one's start, last 16 bytes or end."""
    where = {name: (i + 1) * AT for i, name in enumerate(size)}
    for name, (other, off) in at.items():
        up = -(-size[other] // 16) * 16
        where[name] = where[other] + {"last": max(up - 16, 0), "end": up}.get(off, off)
    return where


def rows_bytes(b, N, xdt):
    return sk.sketch_int8_layout(sk.Int8Params(b, N, 1)).bytes if xdt == sk.INT8_ROWS else b * N * (4 if xdt == sk.F32 else 2)


def matmul(M, N, b, xdt, **at):
    p = sk.Int8Params(M, N, 1)
    need = sk.sketch_int8_workspace_bytes(p, b, xdt, sk.F32)
    where = place(dict(buf=sk.sketch_int8_layout(p).bytes, X=rows_bytes(b, N, xdt), Y=b * M * 4, ws=need), at)
    return sk.lib().sketch_int8_matmul(ctypes.byref(p), vp(where["buf"]), vp(where["X"]), xdt, b, vp(where["Y"]), sk.F32,
                                       vp(where["ws"]), need, None)


@pytest.mark.parametrize("xdt", [sk.F32, sk.BF16, sk.F16, sk.INT8_ROWS])
@pytest.mark.parametrize("M,N", [(256, 256), (300, 1000), (20000, 1000)])
@pytest.mark.parametrize("b", [1, 4, 16, 17, 200])
def test_products(M, N, b, xdt):
    encoded_first = xdt != sk.INT8_ROWS and b > sk.INT8_TOKENS
    need = sk.sketch_int8_workspace_bytes(sk.Int8Params(M, N, 1), b, xdt, sk.F32)
    assert matmul(M, N, b, xdt) != sk.EINVAL
    for off in (0, 16, "last"):
        got = matmul(M, N, b, xdt, Y=("X", off))
        assert (got != sk.EINVAL) if encoded_first else (got == sk.EINVAL), off
        assert matmul(M, N, b, xdt, Y=("buf", off)) == sk.EINVAL
        for other in ("X", "Y", "buf") if need else ():
            assert matmul(M, N, b, xdt, ws=(other, off)) == sk.EINVAL, other
    assert matmul(M, N, b, xdt, Y=("X", "end")) != sk.EINVAL
    assert matmul(M, N, b, xdt, X=("Y", "end")) != sk.EINVAL
    assert matmul(M, N, b, xdt, ws=("Y", "end"), X=("buf", "end")) != sk.EINVAL


def group(M, N, E, terms, xrows, xdt, bits, index, **at):
    p = sk.Int8Params(M, N, E)
    need = sk.sketch_int8_group_workspace_bytes(p, terms, xrows, xdt, sk.F32)
    where = place(dict(buf=E * sk.sketch_int8_layout(p).bytes, X=rows_bytes(xrows, N, xdt), Y=terms * M * 4, ws=need,
                       counts=E * bits // 8, rows=terms * bits // 8), at)
    g = sk.Int8Groups(terms, where["counts"], where["rows"] if index else None, bits, bits)
    return sk.lib().sketch_int8_matmul_group(ctypes.byref(p), vp(where["buf"]), vp(where["X"]), xdt, xrows, ctypes.byref(g),
                                             vp(where["Y"]), sk.F32, vp(where["ws"]), need, None)


@pytest.mark.parametrize("xdt", [sk.F32, sk.BF16, sk.INT8_ROWS])
@pytest.mark.parametrize("terms", [3, 40, 700])
@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("index", [False, True])
def test_groups(xdt, terms, bits, index):
    args = (130, 300, 6, terms, terms, xdt, bits, index)
    need = sk.sketch_int8_group_workspace_bytes(sk.Int8Params(130, 300, 6), terms, terms, xdt, sk.F32)
    assert group(*args) != sk.EINVAL
    others = ("buf", "X", "counts") + (("rows",) if index else ())
    for off in (0, "last"):
        for other in others:
            assert group(*args, Y=(other, off)) == sk.EINVAL, other
        for other in others + ("Y",) if need else ():
            assert group(*args, ws=(other, off)) == sk.EINVAL, other
    assert group(*args, Y=("X", "end")) != sk.EINVAL
    assert group(*args, counts=("rows", "end")) != sk.EINVAL
