"""Rows that have no columns at all are refused like rows of other lengths (no GPU)."""
import pytest
import torch

sk = pytest.importorskip("sub_bit_weight_sketch_amd")


@pytest.mark.parametrize("shape", [(), (2, 199), (199,), (2, 2, 200)])
def test_products_refuse_rows_of_another_shape(shape):
    X = torch.zeros(shape)
    with pytest.raises(ValueError, match="X must have 200 columns"):
        sk.int8_matmul(sk.Int8Tables(4, 200, None, "cpu"), X)
    with pytest.raises(ValueError, match="X must have 200 columns"):
        sk.fp8_matmul(sk.Fp8Tables(4, 200, 128, None, "cpu"), X)
