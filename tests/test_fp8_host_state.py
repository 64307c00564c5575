"""Sizes of tables and layers cannot be changed by a caller, neither their own nor
those of others of the same shape (no GPU)."""
import pytest

sk = pytest.importorskip("sub_bit_weight_sketch_amd")


def fields(s):
    return {n: getattr(s, n) for n, _ in s._fields_}


def test_parameters_and_layouts_are_copies():
    t, other = (sk.Fp8Tables(70, 300, 128, None, "cpu") for _ in range(2))
    params, layout = fields(t.params), fields(t.layout)
    p, s = t.params, t.layout
    p.M, p.N, p.count, s.ld, s.bytes, s.scales_offset = 7, 8, 9, 1, 2, 3
    for x in (t, other, sk.Fp8Tables(70, 300, 128, None, "cpu")):
        assert fields(x.params) == params and fields(x.layout) == layout
        assert x.codes().stride() == (384, 1) and x.codes().shape == (70, 300)


@pytest.mark.parametrize("name", ["M", "N", "block_rows", "count", "device", "params", "layout", "shape"])
def test_sizes_of_tables_are_read_only(name):
    t = sk.Fp8Tables(70, 300, 1, 2, "cpu")
    with pytest.raises(AttributeError):
        setattr(t, name, getattr(t, name))


def test_parameters_of_a_layer_are_a_copy():
    layer = sk.MoE.__new__(sk.MoE)
    layer._params, layer._ws = sk.MoEParams(256, 128, 8, 2, 1, sk.F32), {}
    need = sk.sketch_moe_workspace_bytes(layer._params, 9)
    layer.params.topk = 8
    assert layer.params.topk == 2 and layer._workspace_bytes(9) == need
    with pytest.raises(AttributeError):
        layer.params = sk.MoEParams(256, 128, 8, 4, 1, sk.F32)


def test_a_stack_keeps_its_count():
    t = sk.Fp8Tables(5, 130, 128, 3, "cpu")
    assert (t.count, t.shape, t.params.count) == (3, (3, 5, 130), 3)
    assert t.buf.numel() == 3 * t.layout.bytes
