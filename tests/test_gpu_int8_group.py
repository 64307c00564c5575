"""Products grouped by expert on the GPU against the plain form, bit for bit."""
import numpy as np
import pytest
import torch

import int8_util as u
from gpu_util import dev
from int8_util import DT, ragged, randn

sk = pytest.importorskip("sub_bit_weight_sketch_amd")

pytestmark = pytest.mark.gpu


def experts(E, M, N, seed):
    return sk.int8_encode(randn((E, M, N), seed, 0.1).to(dev()))


def check(w, X, counts, rows=None, y="f32", wide=(False, False), encoded=False, terms=None):
    """counts, rows: lists.  The output starts as random numbers, of which those
    behind the last term have to stay."""
    q, s = u.encode(u.to64(X))
    n = len(rows) if rows is not None else X.shape[0]
    out = randn((n, w.M), 77, 1.0, y).to(dev())
    want = u.group(q, s, rows, counts, *u.table(w), out.cpu())
    kind = [torch.int64 if v else torch.int32 for v in wide]
    c = torch.tensor(counts, dtype=kind[0], device=dev())
    r = torch.tensor(rows, dtype=kind[1], device=dev()) if rows is not None else None
    x = sk.int8_encode(X, check=False) if encoded else X
    got = sk.int8_matmul_group(w, x, c, rows=r, out=out)
    assert got is out
    u.same(got, want)


CASES = [(1, 33, 130, 1), (2, 16, 64, 2), (8, 300, 1000, 3), (8, 256, 512, 16), (8, 130, 257, 40), (64, 96, 200, 42),
         (64, 130, 300, 700), (5, 515, 700, 333), (3, 128, 128, 1000), (512, 40, 64, 100), (512, 17, 130, 3000),
         (100, 64, 256, 257), (65, 64, 128, 200), (4, 1030, 2050, 500), (16, 2816, 512, 90)]


@pytest.mark.parametrize("E,M,N,terms", CASES)
@pytest.mark.parametrize("x,y,encoded", [("bf16", "bf16", False), ("f32", "f32", True), ("f16", "f16", False)])
def test_ragged(E, M, N, terms, x, y, encoded):
    w = experts(E, M, N, E + M)
    for seed in range(3):
        check(w, randn((terms, N), seed, 1.0, x).to(dev()), ragged(E, terms, seed + terms), y=y, encoded=encoded,
              wide=(seed == 1, False))


@pytest.mark.parametrize("E,M,N,T,k", [(8, 300, 1000, 1, 2), (8, 300, 600, 9, 2), (64, 130, 300, 7, 6), (64, 100, 300, 130, 6),
                                       (4, 515, 700, 300, 3)])
@pytest.mark.parametrize("encoded", [False, True])
def test_rows_of_tokens(E, M, N, T, k, encoded):
    """Each token at k experts: its row is taken k times."""
    g = np.random.default_rng(T)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).ravel()
    rows = (np.argsort(ids, kind="stable") // k).tolist()
    counts = np.bincount(ids, minlength=E).tolist()
    w = experts(E, M, N, 4)
    X = randn((T, N), 3, 1.0, "bf16").to(dev())
    for wide in ((False, False), (True, True)):
        check(w, X, counts, rows, "bf16", wide, encoded)


@pytest.mark.parametrize("x", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [1, 1000, 2048, 2100, 4100, 30000, 40000])
def test_few_raw_rows(N, x):
    """Rows that the product encodes itself, at the lengths where it stops to; an expert of one term and one of several."""
    w = experts(5, 70, N, 2)
    for T, counts in ((1, [0, 0, 1, 0, 0]), (7, [0, 1, 4, 1, 1]), (30, [17, 0, 5, 1, 2])):
        X = randn((T, N), T, 1.0, x).to(dev())
        X[0, 0] = float("nan")
        check(w, X, counts)
        g = np.random.default_rng(N)
        rows = g.integers(0, T, sum(counts) + 3)
        rows[0] = T
        check(w, X, counts, rows.tolist(), "bf16", (True, True))


@pytest.mark.parametrize("terms", [1, 15, 16, 17, 31, 32, 33, 64, 65, 128, 129, 256, 300])
@pytest.mark.parametrize("where", [0, 2, 3])
def test_one_expert_has_everything(terms, where):
    counts = [0, 0, 0, 0]
    counts[where] = terms
    check(experts(4, 140, 260, 1), randn((terms, 260), terms, 1.0, "bf16").to(dev()), counts, y="bf16")


@pytest.mark.parametrize("terms", [40, 500])
def test_counts_that_do_not_add_up(terms):
    """Less than the terms (a padded batch: the rest stays), more than the terms
    (cut off), negative ones (zero), none at all, and the largest integers."""
    w = experts(6, 70, 200, 2)
    X = randn((terms, 200), 1).to(dev())
    for counts in ([3, 0, 5, 0, 1, 2], [0] * 6, [terms] * 6, [terms - 3, 2, 2, 2, 2, 2], [-5, 7, -1, 9, -(2 ** 31), 4],
                   [2 ** 31 - 1] * 6, [1, 2 ** 31 - 1, 1, 1, 1, 1]):
        check(w, X, counts)
        check(w, X, counts, wide=(True, False))
    check(w, X, [7, 2 ** 62, 2 ** 62, 2 ** 63 - 1, 1, 1], wide=(True, False))
    check(w, X, [7, -(2 ** 63), 2 ** 32, 3, 1, 1], wide=(True, False))
    check(w, X, [7, 2 ** 32 + 1, 3, 3, 1, 1], wide=(True, False))


@pytest.mark.parametrize("terms", [12, 200])
def test_rows_outside_give_nan(terms):
    w = experts(3, 70, 130, 2)
    X = randn((10, 130), 1).to(dev())
    g = np.random.default_rng(1)
    rows = g.integers(0, 10, terms)
    rows[1], rows[5], rows[7] = -1, 10, 2 ** 31 - 1
    counts = [terms // 2, 1, terms - terms // 2 - 1]
    for wide in (False, True):
        check(w, X, counts, rows.tolist(), wide=(False, wide))
        check(w, X, counts, rows.tolist(), wide=(False, wide), encoded=True)
    rows[1], rows[5], rows[8] = 2 ** 32, 2 ** 32 + 3, -(2 ** 63)
    check(w, X, counts, rows.tolist(), wide=(False, True))


def test_the_same_row_everywhere_and_more_terms_than_rows():
    w = experts(4, 64, 128, 2)
    X = randn((3, 128), 1, 1.0, "f16").to(dev())
    check(w, X, [100, 0, 60, 40], [1] * 200, "f16")
    check(w, X, [100, 0, 60, 40], ([0, 1, 2] * 67)[:200], "f16")


def test_nan_rows_and_experts_stay_where_they_are():
    w = experts(4, 70, 200, 3)
    X = randn((50, 200), 1, 1.0, "bf16").to(dev())
    X[4, 3] = float("nan")
    X[30, 0] = float("inf")
    w.scales()[2, 5] = float("nan")
    check(w, X, [10, 15, 20, 5])
    X = randn((300, 200), 1, 1.0, "bf16").to(dev())
    X[4, 3] = float("nan")
    check(w, X, [100, 50, 140, 10])


def test_empty_calls_and_a_single_matrix_of_a_stack():
    w = experts(2, 70, 200, 3)
    c = torch.tensor([0, 0], device=dev())
    assert sk.int8_matmul_group(w, torch.empty(0, 200, device=dev()), c).shape == (0, 70)
    rows = torch.empty(0, dtype=torch.int32, device=dev())
    assert sk.int8_matmul_group(w, torch.zeros(4, 200, device=dev()), c, rows=rows).shape == (0, 70)
    with pytest.raises(sk.SketchError):       # terms, but no row to take
        sk.int8_matmul_group(w, torch.empty(0, 200, device=dev()), c, rows=torch.zeros(3, dtype=torch.int32, device=dev()))


def test_dense_product_is_the_group_of_one():
    w = sk.int8_encode(randn((1, 300, 700), 5, 0.1).to(dev()))
    one = sk.int8_encode(randn((300, 700), 5, 0.1).reshape(300, 700).to(dev()))
    assert torch.equal(one.codes(), w.codes()[0])
    for b in (1, 6, 40, 300):
        X = randn((b, 700), b, 1.0, "bf16").to(dev())
        assert torch.equal(sk.int8_matmul_group(w, X, torch.tensor([b], device=dev())), sk.int8_matmul(one, X))


@pytest.mark.parametrize("terms", [30, 600])
def test_out_may_be_x_and_workspace(terms):
    w = experts(4, 256, 256, 1)
    X = randn((terms, 256), 2).to(dev())
    c = torch.tensor([terms // 2, 0, 5, terms - terms // 2 - 5], device=dev())
    ws = sk.int8_group_workspace_for(w, terms, terms, sk.F32, sk.F32, dev())
    want = sk.int8_matmul_group(w, X, c, workspace=ws)
    sk.int8_matmul_group(w, X, c, out=X, workspace=ws)
    assert torch.equal(X, want)
    if ws is not None:
        with pytest.raises(sk.SketchError) as e:
            sk.int8_matmul_group(w, X, c, workspace=ws[:64])
        assert e.value.code == sk.ESMALL


@pytest.mark.parametrize("T", [3, 200])
def test_in_a_graph_with_new_routes(T):
    """One captured call serves every routing of the same number of terms."""
    E, k = 8, 2
    w = experts(E, 200, 384, 1)
    X = randn((T, 384), 0, 1.0, "bf16").to(dev())
    counts = torch.zeros(E, dtype=torch.int64, device=dev())
    rows = torch.zeros(T * k, dtype=torch.int64, device=dev())
    Y = torch.empty((T * k, 200), device=dev())
    ws = sk.int8_group_workspace_for(w, T * k, T, sk.BF16, sk.F32, dev())

    def route(seed):
        ids = torch.rand(T, E, generator=torch.Generator().manual_seed(seed)).topk(k).indices.flatten()
        rows.copy_(torch.sort(ids, stable=True).indices // k)
        counts.copy_(torch.bincount(ids, minlength=E))
        X.copy_(randn((T, 384), seed, 1.0, "bf16"))

    route(0)
    sk.int8_matmul_group(w, X, counts, rows=rows, out=Y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sk.int8_matmul_group(w, X, counts, rows=rows, out=Y, workspace=ws)
    for i in range(1, 4):
        route(i)
        want = sk.int8_matmul_group(w, X, counts, rows=rows)
        Y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want), i


def test_experts_beyond_4_gib():
    """Experts whose codes lie past 2^32 bytes, and a routing that needs them."""
    E, M, N = 40, 1024, 131071
    w = sk.Int8Tables(M, N, E, dev())
    w.buf.zero_()
    g = torch.Generator(device=dev()).manual_seed(3)
    at = [0, 17, 1023]
    for e in (0, 31, 32, 39):
        w.codes()[e, at] = torch.randint(-127, 128, (3, N), generator=g, device=dev(), dtype=torch.int8)
        w.scales()[e, at] = 1.0
    for terms in (9, 260):
        x = sk.int8_encode(randn((terms, N), terms, 1.0, "bf16").to(dev()))
        counts = [0] * E
        counts[0], counts[31], counts[32], counts[39] = 1, terms // 2, terms - terms // 2 - 2, 1
        Y = sk.int8_matmul_group(w, x, torch.tensor(counts, device=dev()))
        q, s = u.table(x)
        for e, a, b in u.spans(counts, terms):
            qw = w.codes()[e, at].cpu().numpy().astype(np.int64)
            u.same(Y[a:b, at], u.product(q[a:b], s[a:b], qw, np.ones(3, np.float32), "f32"))
        Y[:, at] = 0
        assert not Y.any()


def test_rows_of_x_beyond_4_gib():
    """Terms whose rows of X lie past 2^32 bytes, few and many."""
    R, N, M = 40000, 131071, 40
    x = sk.Int8Tables(R, N, None, dev())
    x.buf.zero_()
    g = torch.Generator(device=dev()).manual_seed(3)
    at = [0, 5, 32766, 32767, 32768, 39000, R - 1]
    x.codes()[at] = torch.randint(-127, 128, (len(at), N), generator=g, device=dev(), dtype=torch.int8)
    x.scales()[at] = torch.rand(len(at), generator=g, device=dev())
    w = sk.int8_tables(torch.randint(-127, 128, (2, M, N), generator=g, device=dev(), dtype=torch.int8),
                       torch.rand(2, M, generator=g, device=dev()))
    for terms in (9, 300, 3000):
        rows = torch.tensor([at[i * i % len(at)] for i in range(terms)], device=dev())
        counts = [terms // 3, terms - terms // 3]
        Y = sk.int8_matmul_group(w, x, torch.tensor(counts, device=dev()), rows=rows)
        for e, a, b in u.spans(counts, terms):
            r = rows[a:b]
            total = torch.matmul(x.codes()[at].double(), w.codes()[e].double().t().contiguous()).float()
            i = torch.tensor([at.index(v) for v in r.tolist()], device=dev())
            assert torch.equal(Y[a:b], total[i] * x.scales()[r][:, None] * w.scales()[e]), terms


# --------------------------------------------------------------------------
# the operators together: a prompt through the experts of a layer
# --------------------------------------------------------------------------

@pytest.mark.parametrize("H,I,E,k,T", [(256, 128, 8, 2, 5), (300, 200, 16, 4, 90), (512, 384, 4, 2, 300)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_experts_of_a_layer(H, I, E, k, T, dt):
    """Router, gate and up side by side, SwiGLU, down, weighted sum.  Against
    float64 on the decoded weights and activations.  Tolerances, relative to an
    output row's size: what the codes of x and h stand for is used on both sides
    (h's as the kernel made them, which test_swiglu checks), so the down products
    differ by the float32 roundings of their values (3 of 2^-24), the weights'
    (2^-24) and the sum of k terms: (k + 4) 2^-24, with the rounding to dt (half a
    step) of each term."""
    g = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=g)
    gate_up = sk.int8_encode((rn(E, 2 * I, H) / H ** 0.5).to(dev()))
    down = sk.int8_encode((rn(E, H, I) / I ** 0.5).to(dev()))
    X = rn(T, H).to(DT[dt]).to(dev())
    logits = rn(T, E).to(dev())
    top, ids = logits.topk(k, dim=1)
    weights = torch.softmax(top, 1)
    order = torch.sort(ids.flatten(), stable=True).indices
    counts = torch.bincount(ids.flatten(), minlength=E)

    gu = sk.int8_matmul_group(gate_up, X, counts, rows=order // k, dtype=DT[dt])
    h = sk.int8_swiglu(gu[:, :I], gu[:, I:])
    d = sk.int8_matmul_group(down, h, counts, dtype=DT[dt])
    back = torch.empty_like(order)
    back[order] = torch.arange(T * k, device=dev())
    Y = (d[back].float().view(T, k, H) * weights[:, :, None]).sum(1)

    # the same experts one by one, from the definitions
    value = lambda t: u.table(t)[0] * u.table(t)[1].astype(np.float64)[..., None]
    q, s = u.encode(u.to64(X))
    x64, gu_w, down_w, h64 = q * s.astype(np.float64)[:, None], value(gate_up), value(down), value(h)
    eps = torch.finfo(DT[dt]).eps / 2 if dt != "f32" else 0.0
    y64 = np.zeros((T, H))
    o, w64 = order.cpu().numpy(), u.to64(weights).reshape(-1)
    bound = np.zeros((T, 1))
    for e, a, b in u.spans(counts.cpu().numpy(), T * k):
        tok = o[a:b] // k
        want = x64[tok] @ gu_w[e].T
        err = np.abs(u.to64(gu)[a:b] - want)
        assert (err <= np.abs(want) * (3 * 2.0 ** -24 + eps) * 1.01 + 1e-12).all()
        dn = h64[a:b] @ down_w[e].T
        contribution = dn * w64[o[a:b]][:, None]
        np.add.at(y64, tok, contribution)
        np.add.at(bound, tok, np.abs(contribution).max(axis=1, keepdims=True))
    assert (np.abs(u.to64(Y) - y64) <= bound * ((k + 4) * 2.0 ** -24 + eps) * 1.01).all()
