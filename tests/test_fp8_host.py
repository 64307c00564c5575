"""Host-side checks of the e4m3 linears and the mixture-of-experts layer (no
GPU): exports, buffer layout, and refusals before anything is enqueued."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import fp8_util as u

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sketch_fp8.h")
vp = ctypes.c_void_p


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sketch_[a-z0-9_]+)\s*\(", text))
    assert names == set(sk.FP8_EXPORTS)
    for n in names:
        assert hasattr(sk.lib(), n) and callable(getattr(sk, n)), n


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "%s"\nsketch_fp8_params p; sketch_moe_params q;\nint main(void) { return SKETCH_FP8_ROWS - 3; }\n'
                   % HEADER)
    assert subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", str(src)]).returncode == 0


def test_plain_form_agrees_with_the_formats():
    """The tests' own oracle: its rounding against torch's e4m3 conversion on
    all finite codes, their midpoints and neighbours, its decoder on every code."""
    bits = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(bits).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    got = u.e4m3_value(bits)
    assert np.array_equal(got[~np.isnan(got)], ref[~np.isnan(ref)]) and np.array_equal(np.isnan(got), np.isnan(ref))
    pos = np.sort(ref[(ref >= 0)])
    mid = (pos[1:] + pos[:-1]) / 2
    probe = np.concatenate([pos, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                            np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64)])
    probe = np.concatenate([probe, -probe])
    want = torch.from_numpy(probe).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(u.e4m3_round(probe), want)


def test_plain_scale_is_the_smallest_that_fits():
    for amax, e in ((448.0, 0), (np.nextafter(448.0, 1e9), 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (0.0, -127),
                    (3e38, 120), (448 * 2.0 ** -127, -127), (2.0 ** -149, -127)):
        assert u.encode(np.array([[amax]]), 1)[1][0, 0] == e + 127, amax


@pytest.mark.parametrize("M,N,rows", [(1, 1, 1), (128, 128, 128), (129, 129, 128), (4096, 11008, 128), (17, 513, 1),
                                      (0, 640, 128)])
def test_layout(M, N, rows):
    s = sk.sketch_fp8_layout(sk.Fp8Params(M, N, rows, 1))
    assert s.ld == u.blocks(N, 128) * 128 and s.col_blocks == u.blocks(N, 128)
    assert s.lds == u.blocks(s.col_blocks, 4) * 4 and s.row_blocks == u.blocks(M, rows)
    assert s.scales_offset == u.blocks(M * s.ld, 256) * 256
    assert s.bytes == u.blocks(s.scales_offset + s.row_blocks * s.lds, 256) * 256


def test_layout_does_not_overflow():
    s = sk.sketch_fp8_layout(sk.Fp8Params(1 << 24, 1 << 20, 128, 1))
    assert s.scales_offset == 1 << 44


@pytest.mark.parametrize("p", [(-1, 64, 128, 1), (1 << 25, 64, 128, 1), (4, 0, 128, 1), (4, (1 << 20) + 1, 128, 1),
                               (4, 64, 64, 1), (4, 64, 0, 1), (4, 64, 128, -1), (4, 64, 128, 65537)])
def test_layout_rejects(p):
    with pytest.raises(sk.SketchError) as e:
        sk.sketch_fp8_layout(sk.Fp8Params(*p))
    assert e.value.code == sk.EINVAL


def test_encode_and_matmul_validate_before_launching():
    sk.sketch_fp8_layout(sk.Fp8Params(1, 1, 1, 1))     # argument types declared
    L, ref = sk.lib(), ctypes.byref
    p = sk.Fp8Params(64, 100, 128, 1)
    assert L.sketch_fp8_encode(ref(p), None, sk.BF16, vp(256), None, None) == sk.EINVAL
    assert L.sketch_fp8_encode(ref(p), vp(264), sk.BF16, vp(256), None, None) == sk.EINVAL
    assert L.sketch_fp8_encode(ref(p), vp(256), sk.BF16, vp(264), None, None) == sk.EINVAL
    assert L.sketch_fp8_encode(ref(p), vp(256), 3, vp(256), None, None) == sk.EINVAL
    assert L.sketch_fp8_encode(ref(p), vp(256), sk.BF16, vp(256), vp(2), None) == sk.EINVAL
    assert L.sketch_fp8_encode(ref(sk.Fp8Params(0, 100, 128, 1)), None, sk.F32, None, None, None) == sk.OK
    n = ctypes.c_size_t()
    assert L.sketch_fp8_workspace_bytes(ref(p), -1, sk.BF16, sk.F32, ref(n)) == sk.EINVAL
    assert L.sketch_fp8_workspace_bytes(ref(p), 4, 4, sk.F32, ref(n)) == sk.EINVAL
    assert L.sketch_fp8_workspace_bytes(ref(p), 4, sk.BF16, sk.F32, None) == sk.EINVAL
    assert L.sketch_fp8_workspace_bytes(ref(sk.Fp8Params(64, 100, 1, 1)), 4, sk.BF16, sk.F32, ref(n)) == sk.EINVAL
    assert L.sketch_fp8_workspace_bytes(ref(sk.Fp8Params(64, 100, 128, 2)), 4, sk.BF16, sk.F32, ref(n)) == sk.EINVAL
    assert L.sketch_fp8_workspace_bytes(ref(p), 0, sk.BF16, sk.F32, ref(n)) == sk.OK and n.value == 0
    big = sk.sketch_fp8_workspace_bytes(p, 4096, sk.BF16, sk.BF16)
    assert L.sketch_fp8_workspace_bytes(ref(p), 4, sk.BF16, 3, ref(n)) == sk.EINVAL
    assert big >= 4096 * 128       # room for the encoded rows at least
    mm = L.sketch_fp8_matmul
    assert mm(ref(p), vp(256), vp(256), sk.BF16, 0, vp(256), sk.F32, None, 0, None) == sk.OK
    assert mm(ref(sk.Fp8Params(0, 100, 128, 1)), None, None, sk.BF16, 4, None, sk.F32, None, 0, None) == sk.OK
    assert mm(ref(p), None, vp(256), sk.BF16, 4, vp(256), sk.F32, vp(256), 1 << 30, None) == sk.EINVAL
    assert mm(ref(p), vp(256), vp(264), sk.BF16, 4, vp(256), sk.F32, vp(256), 1 << 30, None) == sk.EINVAL
    assert mm(ref(p), vp(256), vp(256), sk.BF16, 4, vp(260), sk.F32, vp(256), 1 << 30, None) == sk.EINVAL
    assert mm(ref(p), vp(256), vp(256), sk.BF16, 4096, vp(256), sk.F32, None, 0, None) == sk.EINVAL
    assert mm(ref(p), vp(256), vp(256), sk.BF16, 4096, vp(256), sk.BF16, vp(256), big - 1, None) == sk.ESMALL
    assert mm(ref(p), vp(256), vp(256), sk.BF16, 4, vp(256), 3, vp(256), 1 << 30, None) == sk.EINVAL
    assert mm(ref(p), vp(256), vp(256), 7, 4, vp(256), sk.F32, vp(256), 1 << 30, None) == sk.EINVAL
    huge = sk.Fp8Params(1 << 24, 100, 128, 1)        # more tiles than a grid holds: nothing is enqueued
    assert mm(ref(huge), vp(256), vp(256), sk.BF16, 1 << 24, vp(256), sk.F32, vp(256), (1 << 63) - 1, None) == sk.EINVAL
    assert mm(ref(p), vp(256), vp(256), sk.BF16, 1 << 25, vp(256), sk.F32, vp(256), 1 << 40, None) == sk.EINVAL


def test_moe_validates_before_launching():
    good = dict(H=256, I=128, E=8, topk=2, renorm=1, x_dtype=sk.BF16)
    n = sk.sketch_moe_workspace_bytes(sk.MoEParams(*good.values()), 4)
    assert n > 0 and sk.sketch_moe_workspace_bytes(sk.MoEParams(*good.values()), 0) == 0
    for field, value in (("H", 0), ("I", 0), ("E", 0), ("E", 513), ("topk", 0), ("topk", 9), ("renorm", 2),
                         ("x_dtype", 3), ("H", (1 << 20) + 1)):
        p = sk.MoEParams(*dict(good, **{field: value}).values())
        with pytest.raises(sk.SketchError) as e:
            sk.sketch_moe_workspace_bytes(p, 4)
        assert e.value.code == sk.EINVAL, field
    p, L, ref = sk.MoEParams(*good.values()), sk.lib(), ctypes.byref
    for tokens in (-1, sk.MOE_MAX_TOKENS + 1):
        with pytest.raises(sk.SketchError):
            sk.sketch_moe_workspace_bytes(p, tokens)
    args = [vp(256)] * 5
    assert L.sketch_moe(ref(p), *args, 0, None, None, None, None, 0, None) == sk.OK
    assert L.sketch_moe(ref(p), *args, 4, vp(256), vp(256), vp(256), vp(256), n - 1, None) == sk.ESMALL
    for i in range(9):                       # every pointer: NULL, then misaligned
        for bad in (None, vp(264)):
            q = [vp(256)] * 9
            q[i] = bad
            assert L.sketch_moe(ref(p), *q[:5], 4, *q[5:8], q[8], n, None) == sk.EINVAL, (i, bad)


def test_python_refusals():
    with pytest.raises(ValueError):
        sk.fp8_encode(torch.zeros(4, 4))                 # not on a GPU
    with pytest.raises(ValueError):
        sk.Fp8Tables(4, 4, 128, 0, "cpu")                # an empty stack
    t = sk.Fp8Tables(4, 200, 128, None, "cpu")
    with pytest.raises(ValueError):
        sk.fp8_matmul(t, torch.zeros(2, 199))
    with pytest.raises(ValueError):
        sk.fp8_matmul(sk.Fp8Tables(4, 200, 1, None, "cpu"), torch.zeros(2, 200))
    with pytest.raises(ValueError):
        sk.fp8_matmul(t, sk.Fp8Tables(2, 200, 128, None, "cpu"))
    with pytest.raises(TypeError):
        sk.fp8_matmul(t, torch.zeros(2, 200, dtype=torch.float64))
    with pytest.raises(ValueError):
        sk.fp8_matmul(t, torch.zeros(2, 200))            # both on the host
    with pytest.raises(ValueError):
        sk.fp8_matmul(t, sk.Fp8Tables(2, 200, 1, None, "cpu"))
    with pytest.raises(ValueError):
        sk.fp8_workspace_for(t, 4, sk.F32, sk.F32, "cpu")
    with pytest.raises(ValueError):
        sk.MoE(torch.zeros(8, 64), None, None, None, 2)


def test_a_buffer_stays_its_own():
    """Replacing a buffer would leave the calls with the old one: refused."""
    t = sk.Fp8Tables(4, 200, 128, None, "cpu")
    with pytest.raises(AttributeError):
        t.buf = t.buf.clone()
    for name in ("router", "gate", "up", "down", "topk", "renorm"):
        with pytest.raises(AttributeError):
            setattr(sk.MoE.__new__(sk.MoE), name, None)


def test_views_of_a_buffer():
    t = sk.Fp8Tables(3, 130, 1, 2, "cpu")
    t.buf.copy_(torch.arange(t.buf.numel()).to(torch.uint8))
    flat = np.arange(t.buf.numel()).astype(np.uint8)
    c, s = t.codes().view(torch.uint8).numpy(), t.scales().numpy()
    assert c.shape == (2, 3, 130) and s.shape == (2, 3, 2)
    for m in range(2):
        for r in range(3):
            at = m * t.layout.bytes + r * 256
            assert np.array_equal(c[m, r], flat[at:at + 130])
            at = m * t.layout.bytes + t.layout.scales_offset + r * 4
            assert np.array_equal(s[m, r], flat[at:at + 2])
