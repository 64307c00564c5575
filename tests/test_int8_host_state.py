"""What a table of 8-bit integers starts as (no GPU)."""
import pytest
import torch

sk = pytest.importorskip("sub_bit_weight_sketch_amd")


def dirty_memory(monkeypatch):
    """Memory that nobody has cleared holds anything."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(85))


@pytest.mark.parametrize("M,N,count", [(3, 130, None), (5, 128, None), (2, 1, 4)])
def test_a_table_starts_as_zeros(M, N, count, monkeypatch):
    """The products read the padding of rows, so a table whose codes a caller fills in has to have it zero."""
    dirty_memory(monkeypatch)
    t = sk.Int8Tables(M, N, count, "cpu")
    assert not t.buf.any()
    t.codes().fill_(7)
    t.scales().fill_(1.0)
    rows = torch.stack([t.buf[i * t.layout.bytes:][:M * t.layout.ld].view(M, -1) for i in range(count or 1)])
    assert (rows[:, :, :N] == 7).all() and not rows[:, :, N:].any()


def test_a_given_buffer_keeps_its_bytes():
    n = sk.sketch_int8_layout(sk.Int8Params(3, 130, 1)).bytes
    buf = torch.arange(n).to(torch.uint8)
    t = sk.Int8Tables(3, 130, None, "cpu", buf)
    assert t.buf.data_ptr() == buf.data_ptr() and torch.equal(t.buf, torch.arange(n).to(torch.uint8))
