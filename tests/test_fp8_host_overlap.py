"""Buffers of one call that share memory are refused before anything is enqueued
(no GPU: a call that is not refused fails at its launch, with another code)."""
import ctypes

import pytest

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

vp = ctypes.c_void_p
AT = 1 << 32               # buffers lie at multiples of this


def matmul(M, N, b, xdt, **at):
    """sketch_fp8_matmul with its buffers apart, but for those that `at` places."""
    p = sk.Fp8Params(M, N, 128, 1)
    s = sk.sketch_fp8_layout(p)                        # argument types declared
    need = sk.sketch_fp8_workspace_bytes(p, b, xdt, sk.F32)
    xb = sk.sketch_fp8_layout(sk.Fp8Params(b, N, 1, 1)).bytes if xdt == sk.FP8_ROWS else b * N * (4 if xdt == sk.F32 else 2)
    size = dict(buf=s.bytes, X=xb, Y=b * M * 4, ws=need)
    where = dict(buf=AT, X=2 * AT, Y=3 * AT, ws=4 * AT)
    for name, (other, off) in at.items():              # off: from the other's start, or "last" / "end" of it
        back = {"last": size[other] // 16 * 16 - (0 if size[other] % 16 else 16), "end": -(-size[other] // 16) * 16}
        where[name] = where[other] + back.get(off, off)
    return sk.lib().sketch_fp8_matmul(ctypes.byref(p), vp(where["buf"]), vp(where["X"]), xdt, b, vp(where["Y"]), sk.F32,
                                      vp(where["ws"]), need, None)


@pytest.mark.parametrize("xdt", [sk.F32, sk.BF16, sk.F16, sk.FP8_ROWS])
@pytest.mark.parametrize("M,N", [(256, 256), (300, 1000)])
@pytest.mark.parametrize("b", [1, 4, 5, 16, 17, 200])
def test_products(M, N, b, xdt):
    encoded_first = xdt != sk.FP8_ROWS and b > sk.FP8_TOKENS
    for off in (0, 16, "last"):
        got = matmul(M, N, b, xdt, Y=("X", off))
        assert (got != sk.EINVAL) if encoded_first else (got == sk.EINVAL), off
        assert matmul(M, N, b, xdt, Y=("buf", off)) == sk.EINVAL
        assert matmul(M, N, b, xdt, X=("Y", off)) == got
        if sk.sketch_fp8_workspace_bytes(sk.Fp8Params(M, N, 128, 1), b, xdt, sk.F32):
            for other in ("X", "Y", "buf"):
                assert matmul(M, N, b, xdt, ws=(other, off)) == sk.EINVAL, other
    assert matmul(M, N, b, xdt) != sk.EINVAL           # apart
    assert matmul(M, N, b, xdt, Y=("X", "end")) != sk.EINVAL     # next to each other
    assert matmul(M, N, b, xdt, X=("Y", "end")) != sk.EINVAL


def test_encode():
    for rows in (1, 128):
        p = sk.Fp8Params(100, 200, rows, 3)
        n = 3 * sk.sketch_fp8_layout(p).bytes
        enc = lambda w, buf: sk.lib().sketch_fp8_encode(ctypes.byref(p), vp(w), sk.BF16, vp(buf), None, None)
        for off in (0, 16, n - 16):
            assert enc(AT + off, AT) == sk.EINVAL
        assert enc(AT, AT + 3 * 100 * 200 * 2 - 16) == sk.EINVAL
        assert enc(AT + n, AT) != sk.EINVAL and enc(AT, AT + 3 * 100 * 200 * 2) != sk.EINVAL


@pytest.mark.parametrize("T", [1, 9, 64])
def test_layer(T):
    p = sk.MoEParams(256, 128, 8, 2, 1, sk.F32)
    ws = sk.sketch_moe_workspace_bytes(p, T)
    names = ["router", "gate", "up", "down", "X", "Y", "ids", "weights", "ws"]

    def call(**at):
        where = {n: (i + 1) * AT for i, n in enumerate(names)}
        where.update({n: where[o] for n, o in at.items()})
        w = [vp(where[n]) for n in names]
        return sk.lib().sketch_moe(ctypes.byref(p), *w[:5], T, *w[5:8], w[8], ws, None)

    assert call() != sk.EINVAL and call(Y="X") != sk.EINVAL
    for a in names[5:]:
        for b in names:
            if a != b and (a, b) not in (("Y", "X"),):
                assert call(**{a: b}) == sk.EINVAL, (a, b)
