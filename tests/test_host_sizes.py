"""What tables remember between calls stays bounded, and right (no GPU)."""
import pytest

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

from sub_bit_weight_sketch_amd import fp8, int8  # noqa: E402


def sizes(t, ask, plain):
    """Asks for more sizes than a table remembers, twice over."""
    for _ in range(2):
        for n in range(1, 3000):
            assert ask(n) == plain(n)
            assert len(t._ws) <= 1024
    assert len(t._ws) > 0


def test_workspace_sizes_of_a_weight():
    t = sk.Int8Tables(70, 300, None, "cpu")
    sizes(t, lambda n: int8._workspace_bytes(t, n, sk.BF16, sk.F32),
          lambda n: sk.sketch_int8_workspace_bytes(t.params, n, sk.BF16, sk.F32))
    t = sk.Fp8Tables(70, 300, 128, None, "cpu")
    sizes(t, lambda n: fp8._workspace_bytes(t, n, sk.BF16, sk.F32),
          lambda n: sk.sketch_fp8_workspace_bytes(t.params, n, sk.BF16, sk.F32))


def test_workspace_sizes_of_a_stack():
    t = sk.Int8Tables(70, 300, 4, "cpu")
    sizes(t, lambda n: int8._group_workspace_bytes(t, 2 * n, n, sk.BF16, sk.F32),
          lambda n: sk.sketch_int8_group_workspace_bytes(t.params, 2 * n, n, sk.BF16, sk.F32))
