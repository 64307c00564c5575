"""A prompt through the experts of a layer, as the README has it: right, and
without a wait for the host."""
import os
import re

import pytest
import torch

import int8_util as u
from gpu_util import dev
from int8_util import randn

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def example():
    """The lines of the README from the order of the terms to the last product."""
    text = open(README).read()
    lines = re.search(r"^order = .*?^D = [^\n]*\n", text, re.S | re.M).group(0)
    return compile(lines, "README.md", "exec")


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (9, 64, 6), (200, 8, 2)])
def test_the_readme_s_prompt(T, E, k):
    H, I = 256, 128
    names = dict(sk=sk, torch=torch, E=E, I=I, k=k, X=randn((T, H), T, 1.0, "bf16").to(dev()),
                 gate_up8=sk.int8_encode(randn((E, 2 * I, H), 2, H ** -0.5).to(dev())),
                 down8=sk.int8_encode(randn((E, H, I), 3, I ** -0.5).to(dev())),
                 ids=torch.rand(T, E, generator=torch.Generator().manual_seed(T)).topk(k).indices.to(dev()))
    exec(example(), names)                    # whatever is made once is made here
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")   # any call that waits for the device raises
    try:
        exec(example(), names)
    finally:
        torch.cuda.set_sync_debug_mode("default")
    ids = names["ids"].cpu().flatten()
    order = torch.argsort(ids, stable=True)
    assert names["counts"].tolist() == torch.bincount(ids, minlength=E).tolist()
    X, D = names["X"], names["D"].cpu()
    for i, term in enumerate(order.tolist()):
        e = int(ids[term])
        row = X[term // k:term // k + 1]
        q, s = u.encode(u.to64(row))
        qw, sw = (v[e] for v in u.table(names["gate_up8"]))
        gu = u.product(q, s, qw, sw, "bf16").to(dev())
        h = sk.int8_swiglu(gu[:, :I], gu[:, I:])
        qw, sw = (v[e] for v in u.table(names["down8"]))
        u.same(D[i:i + 1], u.product(*u.table(h), qw, sw, "f32"))
