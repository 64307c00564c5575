"""Host-side checks of the 8-bit integer linears (no GPU): exports, buffer
layout, refusals before anything is enqueued, and the tests' own oracle."""
import ctypes
import fractions
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import int8_util as u

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sketch_int8.h")
vp = ctypes.c_void_p


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sketch_[a-z0-9_]+)\s*\(", text))
    assert names == set(sk.INT8_EXPORTS)
    for n in names:
        assert hasattr(sk.lib(), n) and callable(getattr(sk, n)), n


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "%s"\nsketch_int8_params p; sketch_int8_groups q;\n'
                   'int main(void) { return SKETCH_INT8_ROWS - 4; }\n' % HEADER)
    assert subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", str(src)]).returncode == 0


def test_plain_codes_are_the_nearest_integers():
    """The oracle's codes against rational arithmetic: random values of every
    type, exact middles, and neighbours of middles."""
    g = np.random.default_rng(1)
    rows = [u.to64(u.randn((1, 200), i, 2.0 ** g.integers(-20, 20), dt))[0] for i, dt in enumerate(["f32", "bf16", "f16"] * 4)]
    middles = (np.arange(127) + 0.5) / 127 * 1.984375      # 127 / 64: middles are exact
    near = [np.nextafter(middles.astype(np.float32), np.float32(v)).astype(np.float64) for v in (0, 9)]
    rows.append(np.concatenate([[1.984375], middles, *near, -middles]))
    rows.append(np.concatenate([[2.0 ** -149 * 254], 2.0 ** -149 * np.arange(254), [-(2.0 ** -149)]]))
    for x in rows:
        x = x.astype(np.float32).astype(np.float64)
        code, scale = u.encode(x[None, :])
        amax = fractions.Fraction(np.abs(x).max())
        want = [round(127 * fractions.Fraction(v) / amax) for v in x]      # ties to even
        assert code[0].tolist() == want
        assert scale[0] == np.float32(np.abs(x).max() / 127.0)


@pytest.mark.parametrize("M,N", [(1, 1), (128, 128), (129, 129), (4096, 11008), (17, 513), (0, 640)])
def test_layout(M, N):
    s = sk.sketch_int8_layout(sk.Int8Params(M, N, 1))
    assert s.ld == -(-N // 128) * 128
    assert s.scales_offset == -(-(M * s.ld) // 256) * 256
    assert s.bytes == -(-(s.scales_offset + 4 * M) // 256) * 256


def test_layout_does_not_overflow():
    s = sk.sketch_int8_layout(sk.Int8Params(1 << 24, 131071, 1))
    assert s.scales_offset == 1 << 41


@pytest.mark.parametrize("p", [(-1, 64, 1), ((1 << 24) + 1, 64, 1), (4, 0, 1), (4, 131072, 1), (4, 64, -1), (4, 64, 65537)])
def test_layout_rejects(p):
    with pytest.raises(sk.SketchError) as e:
        sk.sketch_int8_layout(sk.Int8Params(*p))
    assert e.value.code == sk.EINVAL


def test_longest_sum_fits():
    """Codes of -128 on both sides, as a buffer from elsewhere may hold them."""
    assert 128 * 128 * sk.INT8_MAX_N < 2 ** 31


def lib():
    sk.sketch_int8_layout(sk.Int8Params(1, 1, 1))      # argument types declared
    return sk.lib()


def test_encode_validates_before_launching():
    L, ref, p = lib(), ctypes.byref, sk.Int8Params(64, 100, 1)
    enc = L.sketch_int8_encode
    assert enc(ref(p), None, sk.BF16, 100, vp(256), None, None) == sk.EINVAL
    assert enc(ref(p), vp(257), sk.BF16, 100, vp(1 << 20), None, None) == sk.EINVAL     # not aligned to its element
    assert enc(ref(p), vp(258), sk.F32, 100, vp(1 << 20), None, None) == sk.EINVAL
    assert enc(ref(p), vp(256), sk.BF16, 100, vp((1 << 20) + 8), None, None) == sk.EINVAL
    assert enc(ref(p), vp(256), sk.BF16, 100, None, None, None) == sk.EINVAL
    assert enc(ref(p), vp(256), 3, 100, vp(1 << 20), None, None) == sk.EINVAL
    assert enc(ref(p), vp(256), sk.BF16, 99, vp(1 << 20), None, None) == sk.EINVAL
    assert enc(ref(p), vp(256), sk.BF16, 1 << 62, vp(1 << 20), None, None) == sk.EINVAL
    assert enc(ref(p), vp(256), sk.BF16, 100, vp(1 << 20), vp(2), None) == sk.EINVAL
    assert enc(ref(sk.Int8Params(0, 100, 1)), None, sk.F32, 100, None, None, None) == sk.OK
    for at in (256, 256 + 64 * 128):                                                  # shares memory with the buffer
        assert enc(ref(p), vp(256), sk.F32, 100, vp(at), None, None) == sk.EINVAL
    assert enc(ref(p), vp(256), sk.F32, 1 << 20, vp(256 + (1 << 22)), None, None) == sk.EINVAL   # a row of W behind buf


def test_swiglu_validates_before_launching():
    L, ref, p = lib(), ctypes.byref, sk.Int8Params(64, 100, 1)
    go = lambda g=1 << 20, lg=200, up=(1 << 20) + 200, lu=200, dt=sk.BF16, buf=1 << 24, st=None, p=p: L.sketch_int8_swiglu(
        ref(p), vp(g), lg, vp(up), lu, dt, vp(buf), vp(st), None)
    for bad in (dict(g=None), dict(up=None), dict(buf=None), dict(g=(1 << 20) + 1), dict(up=(1 << 20) + 1), dict(lg=99),
                dict(lu=99), dict(lu=1 << 62), dict(dt=3), dict(buf=(1 << 24) + 8), dict(st=2), dict(p=sk.Int8Params(64, 100, 2)),
                dict(buf=1 << 20), dict(buf=(1 << 20) + 63 * 400), dict(up=(1 << 24) + 64)):
        assert go(**bad) == sk.EINVAL, bad
    assert go(p=sk.Int8Params(0, 100, 1), g=None, up=None, buf=None) == sk.OK


def test_matmul_validates_before_launching():
    L, ref, p = lib(), ctypes.byref, sk.Int8Params(64, 100, 1)
    n = ctypes.c_size_t()
    size = L.sketch_int8_workspace_bytes
    for q, b, xdt, ydt in ((p, -1, sk.BF16, sk.F32), (p, 4, 3, sk.F32), (p, 4, 5, sk.F32), (p, 4, sk.BF16, 3),
                           (p, 4, sk.BF16, sk.INT8_ROWS), (sk.Int8Params(64, 100, 2), 4, sk.BF16, sk.F32),
                           (p, sk.INT8_MAX_M + 1, sk.BF16, sk.F32)):
        assert size(ref(q), b, xdt, ydt, ref(n)) == sk.EINVAL, (b, xdt, ydt)
    assert size(ref(p), 4, sk.BF16, sk.F32, None) == sk.EINVAL
    assert size(ref(p), 0, sk.BF16, sk.F32, ref(n)) == sk.OK and n.value == 0
    big = sk.sketch_int8_workspace_bytes(p, 4096, sk.BF16, sk.BF16)
    assert big >= 4096 * 132       # room for the encoded rows at least
    mm = L.sketch_int8_matmul
    w, x, y, ws = vp(1 << 20), vp(1 << 24), vp(1 << 28), vp(1 << 32)
    assert mm(ref(p), w, x, sk.BF16, 0, y, sk.F32, None, 0, None) == sk.OK
    assert mm(ref(sk.Int8Params(0, 100, 1)), None, None, sk.BF16, 4, None, sk.F32, None, 0, None) == sk.OK
    for bad in ((None, x, y), (w, None, y), (w, x, None), (vp((1 << 20) + 8), x, y), (w, vp((1 << 24) + 8), y),
                (w, x, vp((1 << 28) + 4))):
        assert mm(ref(p), bad[0], bad[1], sk.BF16, 4096, bad[2], sk.F32, ws, 1 << 31, None) == sk.EINVAL
    assert mm(ref(p), w, x, sk.BF16, 4096, y, sk.F32, None, 0, None) == sk.EINVAL
    assert mm(ref(p), w, x, sk.BF16, 4096, y, sk.F32, vp((1 << 32) + 8), 1 << 31, None) == sk.EINVAL
    assert mm(ref(p), w, x, sk.BF16, 4096, y, sk.BF16, ws, big - 1, None) == sk.ESMALL
    assert mm(ref(p), w, x, 3, 4, y, sk.F32, ws, 1 << 30, None) == sk.EINVAL
    assert mm(ref(p), w, x, sk.BF16, 4, y, 3, ws, 1 << 30, None) == sk.EINVAL


def test_group_validates_before_launching():
    L, ref, p = lib(), ctypes.byref, sk.Int8Params(64, 100, 8)
    n = ctypes.c_size_t()
    size = L.sketch_int8_group_workspace_bytes
    for q, terms, xr, xdt, ydt in ((p, -1, 4, sk.BF16, sk.F32), (p, 4, -1, sk.BF16, sk.F32), (p, 4, 4, 3, sk.F32),
                                   (p, 4, 4, sk.BF16, 3), (p, sk.INT8_MAX_M + 1, 4, sk.BF16, sk.F32),
                                   (sk.Int8Params(64, 100, sk.INT8_MAX_EXPERTS + 1), 4, 4, sk.BF16, sk.F32)):
        assert size(ref(q), terms, xr, xdt, ydt, ref(n)) == sk.EINVAL
    assert size(ref(p), 4, 4, sk.BF16, sk.F32, None) == sk.EINVAL
    assert size(ref(p), 0, 4, sk.BF16, sk.F32, ref(n)) == sk.OK and n.value == 0
    need = sk.sketch_int8_group_workspace_bytes(p, 600, 5, sk.BF16, sk.F32)
    base = dict(w=1 << 20, x=1 << 24, xdt=sk.BF16, xr=5, terms=600, counts=1 << 25, cb=32, rows=1 << 26, rb=32, y=1 << 28,
                ydt=sk.F32, ws=1 << 32, wsb=need)

    def go(**change):
        a = dict(base, **change)
        g = sk.Int8Groups(a["terms"], a["counts"], a["rows"], a["cb"], a["rb"])
        return L.sketch_int8_matmul_group(ref(p), vp(a["w"]), vp(a["x"]), a["xdt"], a["xr"], ref(g), vp(a["y"]), a["ydt"],
                                          vp(a["ws"]), a["wsb"], None)

    for bad in (dict(w=None), dict(x=None), dict(y=None), dict(counts=None), dict(ws=None), dict(w=(1 << 20) + 8),
                dict(x=(1 << 24) + 8), dict(y=(1 << 28) + 8), dict(ws=(1 << 32) + 8), dict(counts=(1 << 25) + 2),
                dict(rows=(1 << 26) + 2), dict(cb=64, counts=(1 << 25) + 4), dict(rb=64, rows=(1 << 26) + 4), dict(cb=16),
                dict(rb=16), dict(rows=None), dict(xr=0), dict(xdt=3), dict(ydt=4), dict(terms=-1),
                dict(y=1 << 20), dict(y=1 << 25), dict(y=1 << 26), dict(ws=1 << 20), dict(ws=1 << 24), dict(ws=1 << 25),
                dict(ws=1 << 26), dict(ws=1 << 28), dict(y=1 << 24), dict(xdt=sk.INT8_ROWS, y=1 << 24)):
        assert go(**bad) == sk.EINVAL, bad
    assert go(wsb=need - 1) == sk.ESMALL
    assert go(terms=0, w=None, x=None, y=None, counts=None, rows=None, ws=None) == sk.OK
    assert L.sketch_int8_matmul_group(ref(p), vp(256), vp(256), sk.BF16, 5, None, vp(256), sk.F32, vp(256), need, None) == sk.EINVAL


def test_python_refusals():
    cpu = sk.Int8Tables(4, 200, None, "cpu")
    stack = sk.Int8Tables(4, 200, 3, "cpu")
    counts = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: sk.int8_encode(torch.zeros(4, 4)), lambda: sk.int8_swiglu(torch.zeros(4, 4), torch.zeros(4, 4)),
                 lambda: sk.Int8Tables(4, 4, 0, "cpu"), lambda: sk.int8_tables(torch.zeros(4, 4), torch.zeros(4)),
                 lambda: sk.int8_tables(torch.zeros(4, 4, dtype=torch.int8), torch.zeros(4)),
                 lambda: sk.int8_matmul(cpu, torch.zeros(2, 199)), lambda: sk.int8_matmul(stack, torch.zeros(2, 200)),
                 lambda: sk.int8_matmul(cpu, torch.zeros(2, 2, 200)), lambda: sk.int8_matmul(cpu, stack),
                 lambda: sk.int8_matmul(cpu, torch.zeros(2, 200)),       # both on the host
                 lambda: sk.int8_matmul_group(cpu, torch.zeros(2, 200), counts),
                 lambda: sk.int8_matmul_group(stack, torch.zeros(200), counts),
                 lambda: sk.int8_matmul_group(stack, torch.zeros(2, 199), counts),
                 lambda: sk.int8_matmul_group(stack, torch.zeros(2, 200), counts[:2]),
                 lambda: sk.int8_matmul_group(stack, torch.zeros(2, 200), counts.float()),
                 lambda: sk.int8_matmul_group(stack, torch.zeros(2, 200), counts, rows=torch.zeros(2, 2, dtype=torch.int32)),
                 lambda: sk.int8_matmul_group(stack, torch.zeros(2, 200), counts, rows=torch.zeros(2)),
                 lambda: sk.int8_matmul_group(stack, stack, counts), lambda: sk.int8_matmul_group(stack, torch.zeros(2, 200), counts),
                 lambda: sk.int8_workspace_for(cpu, 4, sk.F32, sk.F32, "cpu"),
                 lambda: sk.int8_group_workspace_for(stack, 4, 4, sk.F32, sk.F32, "cpu"),
                 lambda: sk.Int8Tables(4, 200, None, "cpu", torch.zeros(100, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sk.int8_matmul(cpu, torch.zeros(2, 200, dtype=torch.float64)),
                 lambda: sk.int8_matmul_group(stack, torch.zeros(2, 200, dtype=torch.int32), counts)):
        with pytest.raises(TypeError):
            call()


def test_a_buffer_stays_its_own():
    t = sk.Int8Tables(4, 200, None, "cpu")
    for name in ("M", "N", "count", "buf", "device", "params", "layout"):
        with pytest.raises(AttributeError):
            setattr(t, name, None)
    t.params.M, t.layout.ld = 77, 1
    assert t.params.M == 4 and t.layout.ld == 256


def test_views_of_a_buffer():
    t = sk.Int8Tables(3, 130, 2, "cpu")
    t.buf.copy_(torch.arange(t.buf.numel()).to(torch.uint8))
    flat = np.arange(t.buf.numel()).astype(np.uint8)
    c, s = t.codes().numpy(), t.scales().numpy()
    assert c.shape == (2, 3, 130) and s.shape == (2, 3)
    for m in range(2):
        for r in range(3):
            at = m * t.layout.bytes + r * 256
            assert np.array_equal(c[m, r].view(np.uint8), flat[at:at + 130])
            at = m * t.layout.bytes + t.layout.scales_offset + r * 4
            assert np.array_equal(s[m, r:r + 1].view(np.uint8), flat[at:at + 4])
