"""Host-side checks of the kinds of sums of an e4m3 product (no GPU)."""
import ctypes

import pytest

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

vp = ctypes.c_void_p


def test_y_types():
    sk.sketch_fp8_layout(sk.Fp8Params(1, 1, 1, 1))     # argument types declared
    L, n = sk.lib(), ctypes.c_size_t()
    p = ctypes.byref(sk.Fp8Params(64, 100, 128, 1))
    for y in (sk.F32, sk.BF16, sk.F16, sk.BF16 | sk.FP8_F32_SUMS):
        assert L.sketch_fp8_workspace_bytes(p, 4, sk.BF16, y, ctypes.byref(n)) == sk.OK
    for y in (-1, 3, sk.FP8_F32_SUMS, sk.F16 | sk.FP8_F32_SUMS, sk.BF16 | 512):
        assert L.sketch_fp8_workspace_bytes(p, 4, sk.BF16, y, ctypes.byref(n)) == sk.EINVAL
        assert L.sketch_fp8_matmul(p, vp(256), vp(256), sk.BF16, 4, vp(512), y, vp(1024), 1 << 20, None) == sk.EINVAL


def test_few_rows_of_a_tall_weight_take_small_tiles():
    """17 rows of 28672 outputs: tiles of 64 tokens with K split, whose parts show
    in the workspace, not tiles of 256 tokens (112 us against 59 us)."""
    p = sk.Fp8Params(28672, 8192, 128, 1)
    for b in (17, 32, 64):
        parts = sk.sketch_fp8_workspace_bytes(p, b, sk.FP8_ROWS, sk.F32)
        assert parts >= 2 * 4 * b * 28672 and parts % (4 * b * 28672) < 256
    assert sk.sketch_fp8_workspace_bytes(p, 2048, sk.FP8_ROWS, sk.F32) == 0
