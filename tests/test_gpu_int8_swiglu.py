"""SwiGLU with the encoder of rows at the ends of float32's range, against
extended precision (the rules and tolerances of check_swiglu)."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from int8_util import randn
from test_gpu_int8 import check_swiglu

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu


def both_ways(g, up):
    """Rows to a workgroup each and, among enough others, to a wave each."""
    n = g.shape[0]
    lines = -(-(4 * torch.cuda.get_device_properties(0).multi_processor_count + 1) // n)
    for times in (1, lines):
        a, b = g.repeat(times, 1).to(dev()), up.repeat(times, 1).to(dev())
        t = sk.int8_swiglu(a, b)
        assert torch.equal(t.codes(), t.codes()[:n].repeat(times, 1))
        assert torch.equal(t.scales().view(torch.int32), t.scales()[:n].repeat(times).view(torch.int32))
        check_swiglu(a[:n], b[:n], sk.int8_swiglu(a[:n], b[:n]) if times == 1 else first(t, n))


def first(t, n):
    return sk.int8_tables(t.codes()[:n].contiguous(), t.scales()[:n].contiguous())


@pytest.mark.parametrize("N", [9, 300, 2048])
def test_values_at_the_end_of_float32(N):
    """A largest value whose float32 product is the largest finite number while the
    exact one lies beyond it (the row counts as infinite: codes zero, scale NaN),
    exactly at it, and just below."""
    g, up = randn((3, N), 1), randn((3, N), 2)
    last = float(np.finfo(np.float32).max)
    beyond = float.fromhex("0x1.6719f2p+121")
    assert np.float32(91.25) * np.float32(beyond) == np.float32(last) and 91.25 * beyond > last
    below = float(np.nextafter(np.float32(beyond), np.float32(0)))
    assert 91.25 * below < last
    for row, (a, b) in enumerate(((91.25, beyond), (128.0, last / 128), (91.25, below))):
        g[row, N // 2], up[row, N // 2] = a, b
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    t = sk.int8_swiglu(g.to(dev()), up.to(dev()), status=flags)
    assert torch.isnan(t.scales()).tolist() == [True, False, False] and int(flags) == sk.FLAG_WEIGHT_RANGE
    both_ways(g, up)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [7, 300, 1000, 2048, 3001])
def test_subnormal_gates(N, dt):
    """Gates of 2^-149 to 2^-120 beside an `up` of 1e9 to 1e38, alone, with
    ordinary elements of the same size as their product, and with larger ones."""
    g = np.random.default_rng(N)
    rows = []
    for lo, hi, big in ((-149, -120, 1e38), (-149, -145, 1e20), (-149, -149, 1e38), (-140, -126, 1e30), (-128, -124, 1e9),
                        (-149, -120, 1e9), (-133, -126, 3e38)):
        for mixed in (0, 1, 2):
            sign = g.choice([-1.0, 1.0], N)
            a = sign * np.exp2(g.uniform(lo, hi, N)) * g.uniform(1, 2, N)
            b = big * g.uniform(0.05, 1, N)
            if mixed:                                            # every third element an ordinary one
                size = 2.0 ** hi * big * (1 if mixed == 1 else 50)
                ordinary = np.arange(N) % 3 == 1
                a[ordinary] = g.uniform(0.2, 2, ordinary.sum())
                b[ordinary] = size * g.uniform(0.05, 2, ordinary.sum())
            rows.append((a, b))
    gate, up = (torch.from_numpy(np.stack([r[i] for r in rows]).astype(np.float32)) for i in (0, 1))
    gate, up = (v.to(torch.bfloat16) for v in (gate, up)) if dt == "bf16" else (gate, up)
    both_ways(gate, up)


def test_subnormal_gates_by_hand():
    """Gates that differ in their last bits alone: 127 times their ratios."""
    tiny = 2.0 ** -149
    gate = torch.tensor([[3 * tiny, 4 * tiny, 0.0], [7 * tiny, 9 * tiny, 5 * tiny], [-tiny, 2 * tiny, -3 * tiny]])
    up = torch.tensor([[2.0 ** 127, 2.0 ** 127, 1.0], [1e20, 0.8e20, 1e20], [3e38, 3e38, 3e38]])
    t = sk.int8_swiglu(gate.to(dev()), up.to(dev()))
    assert t.codes().tolist() == [[95, 127, 0], [123, 127, 88], [-42, 85, -127]]
    both_ways(gate, up)
