"""What a table of e4m3 codes starts as (no GPU)."""
import pytest
import torch

sk = pytest.importorskip("sub_bit_weight_sketch_amd")


@pytest.mark.parametrize("M,N,block_rows,count", [(3, 130, 128, None), (5, 130, 1, None), (2, 1, 128, 4)])
def test_a_table_starts_as_zeros(M, N, block_rows, count, monkeypatch):
    """The products read the padding of rows, so a table whose codes and scales a
    caller fills in has to have it zero, whatever its memory held before."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(85))
    t = sk.Fp8Tables(M, N, block_rows, count, "cpu")
    assert not t.buf.any()


def test_a_given_buffer_keeps_its_bytes():
    n = sk.Fp8Tables(3, 130, 128, None, "cpu").buf.numel()
    buf = torch.arange(n).to(torch.uint8)
    t = sk.Fp8Tables(3, 130, 128, None, "cpu", buf)
    assert t.buf.data_ptr() == buf.data_ptr() and torch.equal(t.buf, torch.arange(n).to(torch.uint8))
