"""The mixture-of-experts layer on the GPU against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import fp8_util as u
from gpu_util import dev

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(H, I, E, k, dt, seed, renorm=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    router = (rn(E, H) * 1.5 / H ** 0.5).to(DT[dt])
    gate, up = (sk.fp8_encode((rn(E, I, H) / H ** 0.5).to(dev())) for _ in range(2))
    down = sk.fp8_encode((rn(E, H, I) / I ** 0.5).to(dev()))
    return sk.MoE(router.to(dev()), gate, up, down, k, renorm)


def plain(layer, X):
    p = layer.params
    return u.moe(u.to64(X), u.to64(layer.router), u.table_values(layer.gate), u.table_values(layer.up),
                 u.table_values(layer.down), p.topk, bool(p.renorm))


def check(layer, X, what=""):
    """Experts equal; weights within a few roundings (one to float32, the sums
    in float64); y within six times sqrt(n) * 2^-24 of its row's size, n = H + I
    the terms of the two sums an output goes through (each a float32 random
    walk), plus 16 roundings for silu, the split and the weighted sum."""
    Y, ids, w = sk.moe(layer, X, return_routing=True)
    y, i, wr = plain(layer, X)
    assert np.array_equal(ids.cpu().numpy(), i), what
    assert np.abs(u.to64(w) / wr - 1).max() <= 2 * u.EPS32, what
    size = np.sqrt((y ** 2).mean(axis=1, keepdims=True))
    err = (np.abs(u.to64(Y) - y) / size).max()
    n = layer.params.H + layer.params.I
    assert err <= (6 * np.sqrt(n) + 16) * u.EPS32, (what, err)
    return Y


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,I,E,k,T,renorm", [(1, 1, 1, 1, 1, True), (64, 32, 4, 2, 3, True), (128, 128, 8, 8, 2, False),
                                              (257, 129, 8, 2, 16, True), (512, 256, 64, 6, 7, False),
                                              (130, 700, 16, 4, 33, True), (1000, 333, 5, 3, 64, False),
                                              (256, 128, 512, 16, 5, True), (300, 64, 3, 1, 64, True),
                                              (2049, 150, 8, 2, 4, False), (500, 200, 32, 3, 1, True),
                                              (1500, 130, 4, 2, 2, True), (999, 130, 4, 3, 4, False),
                                              (2048, 2000, 8, 4, 5, True), (1030, 4100, 4, 2, 64, True),
                                              (48, 40, 512, 16, 64, False)])
def test_layer(H, I, E, k, T, renorm, dt):
    layer = make(H, I, E, k, dt, H + I + E, renorm)
    X = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(DT[dt]).to(dev())
    check(layer, X)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 40, 64])
def test_all_tokens_at_one_expert(T):
    """More tokens at one expert than a matrix-core tile has columns."""
    layer = make(256, 192, 4, 1, "bf16", 3)
    layer.router[2] = 1.0
    X = (torch.rand(T, 256, generator=torch.Generator().manual_seed(1)) + 0.5).to(torch.bfloat16).to(dev())
    assert (sk.moe(layer, X, return_routing=True)[1] == 2).all()
    check(layer, X)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [4, 5, 6, 7, 8, 9, 15, 17])
def test_few_tokens_at_an_expert(T, dt):
    """One expert with all tokens, others with the even or the odd ones, about
    the numbers at which activations of several terms change their layout."""
    H, I = 300, 150
    layer = make(H, I, 8, 2, dt, 14)
    X = torch.randn(T, H, generator=torch.Generator().manual_seed(T))
    layer.router[:, :2] = 0
    layer.router[5, 0], layer.router[1, 1], layer.router[6, 1] = 40.0, 30.0, -30.0
    X[:, 0] = 1.0
    X[:, 1] = 1.0 - 2.0 * (torch.arange(T) % 2)
    X = X.to(DT[dt]).to(dev())
    ids = sk.moe(layer, X, return_routing=True)[1].cpu()
    assert (ids[:, 0] == 5).all() and (ids[::2, 1] == 1).all() and (ids[1::2, 1] == 6).all()
    check(layer, X)


def test_each_index_path():
    """Gate, up and down pick single entries, so that every output is one known
    term: y[t][i] = sum_e w_e silu(x[a]) x[b], with a, b known from (e, i).
    Wrong rows, columns, experts or scales would each show up whole."""
    H, I, E, k, T = 384, 300, 6, 3, 20
    g = np.random.default_rng(0)
    pa, pb, pd = (g.integers(0, n, (E, m)) for n, m in ((H, I), (H, I), (I, H)))
    gate, up, down = np.zeros((E, I, H), np.float32), np.zeros((E, I, H), np.float32), np.zeros((E, H, I), np.float32)
    for e in range(E):
        gate[e, np.arange(I), pa[e]] = 2.0 ** (np.arange(I) // 128)
        up[e, np.arange(I), pb[e]] = 2.0 ** e
        down[e, np.arange(H), pd[e]] = 2.0 ** (-(np.arange(H) // 128) - e)
    enc = lambda a: sk.fp8_encode(torch.from_numpy(a).to(dev()))
    router = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32)).to(dev())
    layer = sk.MoE(router, enc(gate), enc(up), enc(down), k)
    x = g.standard_normal((T, H)).astype(np.float32) * 0.5
    Y, ids, w = (u.to64(v) for v in sk.moe(layer, torch.from_numpy(x).to(dev()), return_routing=True))
    x = x.astype(np.float64)
    y, size = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for s in range(k):
            e = int(ids[t, s])
            gv = x[t, pa[e]] * 2.0 ** (np.arange(I) // 128)
            h = gv / (1 + np.exp(-gv)) * x[t, pb[e]] * 2.0 ** e
            term = w[t, s] * h[pd[e]] * 2.0 ** (-(np.arange(H) // 128) - e)
            y[t] += term
            size[t] += np.abs(term)
    # roundings: exp (2 steps), 1 + exp, the division, h, w, w * h and k sums: 8 + k steps of 2^-23
    assert (np.abs(Y - y) <= (8 + k) * 2 * u.EPS32 * size).all()


def test_ties_take_the_lower_expert():
    layer = make(128, 64, 16, 5, "bf16", 4)
    layer.router[:] = layer.router[:1].clone()          # all logits equal
    X = torch.randn(3, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(dev())
    _, ids, w = sk.moe(layer, X, return_routing=True)
    assert (ids.cpu() == torch.arange(5, dtype=torch.int32)).all()
    assert np.abs(u.to64(w) - 0.2).max() <= 0.2 * 2 * u.EPS32
    layer.router[:] = 0                                  # +0 and -0 are equal
    layer.router[::2] = -0.0
    assert (sk.moe(layer, X, return_routing=True)[1].cpu() == torch.arange(5, dtype=torch.int32)).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_tokens_stay_in_their_row(bad, dt):
    layer = make(256, 128, 8, 2, dt, 6)
    X = torch.randn(5, 256, generator=torch.Generator().manual_seed(3)).to(DT[dt]).to(dev())
    Y = sk.moe(layer, X)
    Z = X.clone()
    Z[2, 17] = bad
    Yz, ids, _ = sk.moe(layer, Z, return_routing=True)
    keep = torch.tensor([0, 1, 3, 4], device=dev())
    assert not torch.isfinite(Yz[2]).any()
    assert torch.isfinite(Yz[keep]).all() and (Yz[keep] - Y[keep]).abs().max() <= 1e-5 * Y.abs().max()
    assert ((ids >= 0) & (ids < 8)).all() and int(ids[2, 0]) != int(ids[2, 1])


@pytest.mark.parametrize("code", [0.0, 1.0])
def test_a_nan_scale_in_an_expert(code):
    """The scale byte 255 in one block of an expert's down weight, of its gate
    or up weight: NaN for the tokens that chose it (the outputs of the block,
    or all of them), and for nobody else."""
    H, I, E, T = 300, 200, 4, 20
    g = torch.Generator().manual_seed(12)
    router = torch.randn(E, H, generator=g).to(dev())
    X = torch.randn(T, H, generator=g).to(dev())
    for which in range(3):
        w = [torch.randn(*s, generator=g) for s in ((E, I, H), (E, I, H), (E, H, I))]
        ref = sk.moe(sk.MoE(router, *(sk.fp8_encode(v.to(dev())) for v in w), 1), X)
        w[which][1, 128:256, 128:256] = code
        t = [sk.fp8_encode(v.to(dev())) for v in w]
        t[which].scales()[1, 1, 1] = 255
        Y, ids, _ = sk.moe(sk.MoE(router, *t, 1), X, return_routing=True)
        hit = ids[:, 0] == 1
        assert 0 < int(hit.sum()) < T
        cols = slice(128, 256) if which == 2 else slice(None)
        assert torch.isnan(Y[hit][:, cols]).all() and torch.equal(Y[~hit], ref[~hit])
        if which == 2:
            assert torch.equal(Y[hit][:, :128], ref[hit][:, :128]) and torch.equal(Y[hit][:, 256:], ref[hit][:, 256:])


@pytest.mark.parametrize("byte,scale", [(0, 2.0 ** -127), (247, 2.0 ** 120)])
def test_far_scales_in_an_expert(byte, scale):
    """Gate and up as ordinary, down at the ends of the scales: the result of
    ones there, scaled by a power of two (the sums are the same, unless they
    leave float32's normal range: h is made large, or small, enough)."""
    H, I, E, T = 256, 128, 2, 5
    g = torch.Generator().manual_seed(13)
    router = torch.randn(E, H, generator=g).to(dev())
    X = torch.randn(T, H, generator=g).to(dev())
    gate = sk.fp8_encode((torch.randn(E, I, H, generator=g) / 16).to(dev()))
    lift = 2.0 ** 60 if scale < 1 else 2.0 ** -60
    up = sk.fp8_encode((torch.randn(E, I, H, generator=g) * lift).to(dev()))
    codes = (torch.randint(1, 8, (E, H, I), generator=g) * 2).float().to(dev()).to(torch.float8_e4m3fn)
    s = torch.full((E, 2, 1), 127, dtype=torch.uint8, device=dev())
    one = sk.moe(sk.MoE(router, gate, up, sk.fp8_tables(codes, s), 1), X)
    far = sk.moe(sk.MoE(router, gate, up, sk.fp8_tables(codes, torch.full_like(s, byte)), 1), X)
    assert torch.equal(far.double(), one.double() * scale)


def test_repeats_are_identical_and_streams_do_not_mix():
    layer = make(512, 384, 8, 2, "bf16", 7)
    g = torch.Generator().manual_seed(4)
    Xs = [torch.randn(11, 512, generator=g).to(torch.bfloat16).to(dev()) for _ in range(4)]
    ref = [sk.moe(layer, X) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    for _ in range(3):
        outs = []
        for X, s in zip(Xs, streams):
            with torch.cuda.stream(s):
                outs.append(sk.moe(layer, X))
        torch.cuda.synchronize()
        for a, b in zip(outs, ref):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 9, 40])
def test_captured_and_replayed(T):
    """One workspace, two graphs and eager calls in turn."""
    layer = make(300, 200, 8, 2, "f16", 8)
    g = torch.Generator().manual_seed(5)
    Xs = [torch.randn(T, 300, generator=g).to(torch.float16).to(dev()) for _ in range(3)]
    ref = [sk.moe(layer, X) for X in Xs]
    ws = layer.workspace_for(T)
    graphs = []
    for _ in range(2):
        x, Y = Xs[0].clone(), torch.empty(T, 300, device=dev())
        sk.moe(layer, x, out=Y, workspace=ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sk.moe(layer, x, out=Y, workspace=ws)
        graphs.append((gr, x, Y))
    for i in (0, 1, 2, 1):
        for gr, x, Y in graphs:
            x.copy_(Xs[i])
            Y.fill_(float("nan"))
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(Y, ref[i])
            assert torch.equal(sk.moe(layer, Xs[i]), ref[i])


def test_experts_beyond_32_bits():
    """The last of 64 experts of 67 MB lies beyond 4 GiB; all others are zero."""
    H = I = 8192
    E = 64
    g = torch.Generator(device=dev()).manual_seed(2)
    stacks, last = [], []
    for _ in range(3):
        w = torch.randn((8192, 8192), generator=g, device=dev()) / 90
        one = sk.fp8_encode(w)
        t = sk.Fp8Tables(8192, 8192, 128, E, dev())
        t.buf.zero_()
        t.buf[-one.layout.bytes:] = one.buf
        stacks.append(t)
        last.append(one)
    router = torch.zeros((E, H), device=dev())
    router[-1] = 1.0
    X = torch.rand((3, H), generator=g, device=dev())
    Y, ids, w = sk.moe(sk.MoE(router, *stacks, 2), X, return_routing=True)
    assert (ids[:, 0] == E - 1).all() and (ids[:, 1] == 0).all()
    val = [t.codes().double() * torch.exp2(t.scales().double() - 127).repeat_interleave(128, 0).repeat_interleave(128, 1)
           for t in last]
    gv, uv = X.double() @ val[0].t(), X.double() @ val[1].t()
    want = w[:, :1].double() * ((gv * torch.sigmoid(gv) * uv) @ val[2].t())
    # as in check(): the walks of two float32 sums, on the size of a row
    size = want.square().mean(1, keepdim=True).sqrt()
    assert ((Y - want).abs() / size).max() <= (6 * np.sqrt(H + I) + 16) * u.EPS32


def test_strided_and_in_place():
    """Rows of a wider tensor, a misaligned router, and the output written
    over the tokens: all of x is read before any of y is written."""
    H = 200
    layer = make(H, 130, 8, 2, "f32", 15)
    g = torch.Generator().manual_seed(16)
    for T in (2, 30):
        wide = torch.randn(T, 2 * H, generator=g).to(dev())
        X = wide[:, 1:H + 1]
        ref = sk.moe(layer, X.contiguous())
        assert torch.equal(sk.moe(layer, X), ref)
        off = torch.cat([torch.zeros(1, device=dev()), layer.router.flatten()])[1:].view(8, H)
        assert off.data_ptr() % 16 != 0
        assert torch.equal(sk.moe(sk.MoE(off, layer.gate, layer.up, layer.down, 2), X), ref)
        Y = X.contiguous()
        assert sk.moe(layer, Y, out=Y) is Y and torch.equal(Y, ref)


def test_refusals():
    layer = make(128, 64, 8, 2, "bf16", 9)
    X = torch.zeros(4, 128, dtype=torch.bfloat16, device=dev())
    for bad in (X[:, :100], X.float(), X.cpu(), X[0]):
        with pytest.raises(ValueError):
            sk.moe(layer, bad)
    with pytest.raises(sk.SketchError):
        sk.moe(layer, torch.zeros(65, 128, dtype=torch.bfloat16, device=dev()))
    assert sk.moe(layer, X[:0]).shape == (0, 128)
    with pytest.raises(ValueError):
        sk.MoE(layer.router, layer.gate, layer.up, layer.gate, 2)
    with pytest.raises(sk.SketchError):
        sk.MoE(layer.router, layer.gate, layer.up, layer.down, 9)
    with pytest.raises(sk.SketchError):
        sk.moe(layer, X, workspace=torch.empty(256, dtype=torch.uint8, device=dev()))


def test_a_block_of_a_model():
    """The operators as a model runs them: a sketched projection, an 8-bit one
    and the layer of experts, on the same tokens, in one captured step."""
    H, T = 256, 6
    g = torch.Generator().manual_seed(10)
    W = torch.randn(H, H, generator=g) * 0.06
    sketched = sk.encode(W.to(torch.bfloat16).to(dev()), bpw=4.0)
    fp8 = sk.fp8_encode(W.to(dev()))
    layer = make(H, 384, 8, 2, "f32", 11)
    x = torch.randn(T, H, generator=g).to(dev())
    sk.matmul(sketched, x), sk.fp8_matmul(fp8, x), sk.moe(layer, x)

    def step():
        a = sk.matmul(sketched, x)
        b = sk.fp8_matmul(fp8, a)
        return a, b, sk.moe(layer, b)

    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        a, b, y = step()
    for seed in (1, 2, 3):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)))
        gr.replay()
        torch.cuda.synchronize()
        for got, want in zip((a, b, y), step()):
            assert torch.equal(got, want)
        bv = u.encoded(u.to64(a), 1) @ u.table_values(fp8).T
        assert np.abs(u.to64(b) - bv).max() <= 6 * np.sqrt(H) * u.EPS32 * np.abs(bv).max()
        yv, _, _ = plain(layer, b)
        assert np.abs(u.to64(y) - yv).max() <= (6 * np.sqrt(H + 384) + 16) * u.EPS32 * np.abs(yv).max()
