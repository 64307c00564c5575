"""Outputs in the memory of the tokens: as if they had memory of their own."""
import pytest
import torch

from gpu_util import dev

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,b", [(256, 1), (8192, 1), (4096, 2), (8192, 4), (4096, 5), (1000, 16), (4096, 17), (1024, 200)])
def test_a_product_in_place(N, b, dt):
    g = torch.Generator(device=dev()).manual_seed(N + b)
    t = sk.fp8_encode(torch.randn((N, N), generator=g, device=dev()))
    x = torch.randn((b + 3, N), generator=g, device=dev()).to(DT[dt])
    want = sk.fp8_matmul(t, x[1:b + 1].clone(), dtype=DT[dt])
    for to in (1, 0, 3):                     # the same rows, and ones that some of X's share
        y = x.clone()
        got = sk.fp8_matmul(t, y[1:b + 1], out=y[to:to + b])
        assert torch.equal(got, want) and got.data_ptr() == y[to].data_ptr()
        keep = [i for i in range(b + 3) if not to <= i < to + b]
        assert torch.equal(y[keep], x[keep])
    y = x.clone()
    sk.fp8_matmul(t, y[1], out=y[1])
    assert torch.equal(y[1], sk.fp8_matmul(t, x[1].clone(), dtype=DT[dt]))


def test_captured_in_place():
    """x <- W x, three times in a graph, from the same memory each time."""
    N, b = 512, 3
    g = torch.Generator(device=dev()).manual_seed(1)
    t = sk.fp8_encode(torch.randn((N, N), generator=g, device=dev()) / N ** 0.5)
    x0 = torch.randn((b, N), generator=g, device=dev())
    want = x0
    for _ in range(3):
        want = sk.fp8_matmul(t, want)
    x = x0.clone()
    sk.fp8_matmul(t, x, out=x)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        for _ in range(3):
            sk.fp8_matmul(t, x, out=x)
    for _ in range(3):
        x.copy_(x0)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want) and torch.equal(x, sk.fp8_matmul(t, sk.fp8_matmul(t, sk.fp8_matmul(t, x0))))


def test_encoded_rows_in_the_outputs_memory_are_refused():
    t = sk.fp8_encode(torch.randn((256, 256), device=dev()))
    for b in (3, 9, 40):
        x = torch.randn((b, 256), device=dev())
        memory = torch.zeros(b * 256 * 4 + 4096, dtype=torch.uint8, device=dev())
        rows = sk.Fp8Tables(b, 256, 1, None, dev(), memory)
        sk.sketch_fp8_encode(rows.params, x, rows.buf)
        with pytest.raises(sk.SketchError) as e:
            sk.fp8_matmul(t, rows, out=memory[:b * 1024].view(torch.float32).view(b, 256))
        assert e.value.code == sk.EINVAL
        with pytest.raises(sk.SketchError) as e:
            sk.fp8_matmul(t, rows, out=t.buf[:b * 512].view(torch.bfloat16).view(b, 256))
        assert e.value.code == sk.EINVAL
