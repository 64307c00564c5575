"""The operators of a prompt captured together into a graph: gate and up, SwiGLU,
down, replayed with new tokens and routes beside the program's own work."""
import pytest
import torch

from gpu_util import dev
from int8_util import randn

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 7, 150])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_prompt_in_a_graph(T, dt):
    E, k, H, I = 8, 2, 384, 200
    gate_up = sk.int8_encode(randn((E, 2 * I, H), 1, H ** -0.5).to(dev()))
    down = sk.int8_encode(randn((E, H, I), 2, I ** -0.5).to(dev()))
    X = randn((T, H), 0, 1.0, dt).to(dev())
    counts = torch.zeros(E, dtype=torch.int64, device=dev())
    rows = torch.zeros(T * k, dtype=torch.int64, device=dev())
    flags = torch.zeros(1, dtype=torch.int32, device=dev())

    def route(seed):
        ids = torch.rand(T, E, generator=torch.Generator().manual_seed(seed)).topk(k).indices.flatten()
        rows.copy_(torch.sort(ids, stable=True).indices // k)
        counts.copy_(torch.bincount(ids, minlength=E))
        X.copy_(randn((T, H), seed, 1.0, dt))

    def prompt():
        gu = sk.int8_matmul_group(gate_up, X, counts, rows=rows, dtype=X.dtype)
        h = sk.int8_swiglu(gu[:, :I], gu[:, I:], status=flags)
        return sk.int8_matmul_group(down, h, counts), h

    route(0)
    prompt()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D, h = prompt()
    for i in range(1, 5):
        route(i)
        if i == 3:
            X[T // 2, 5] = float("nan")
        flags.zero_()
        want, want_h = prompt()
        want_flags = int(flags)
        D.fill_(7.0)
        flags.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D.view(torch.int32), want.view(torch.int32)), i
        assert torch.equal(h.codes(), want_h.codes()), i
        assert int(flags) == want_flags == (sk.FLAG_WEIGHT_RANGE if i == 3 else 0)
