"""Operators on 8-bit integers: what they compute and how they are timed.

Four operators, on matrices whose rows (a weight's output channels, a batch's
tokens) are integer codes -127..127 with one float32 scale each:

  encode  X [M, N] -> codes [M, N] (int8) and scales [M]
  swiglu  gate, up [M, N] -> codes and scales of h = silu(gate) * up
  matmul  Y = X8 . W8^T, W8 an encoded weight, X8 the rows of X encoded on the
          way in; Y float32, bfloat16 or binary16
  group   the same for a stack of weights, one for each expert: the terms (a
          token at one of its experts) stand in the order of their experts,
          counts[e] of them for expert e; term i multiplies row rows[i] of X, or
          row i of rows that are encoded already.  Rows of Y behind the last
          term are left as they were

The scale of a row is its largest magnitude over 127, rounded to float32; a
code is the integer next to 127 x / (largest magnitude), ties to even.  Sums of
products of codes are exact.  silu(g) = g / (1 + exp(-g)).

With ``own`` false, ``run`` computes in elementary torch operations (the codes
in 64 bits, as they decide between neighbouring integers); with ``own`` true it
calls the library.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the largest linear of the benchmark, encoded once while a model is loaded, beyond the last-level cache
        {"name": "encode_w_mlp_70b", "op": "encode", "M": 28672, "N": 8192, "dt": "bf16", "w": True},
        # activations of a prompt, an odd number of tokens and of columns
        {"name": "encode_rows_odd", "op": "encode", "M": 517, "N": 4001, "dt": "f32", "w": False},
        # a few decode tokens between the two products of an MLP: latency alone
        {"name": "swiglu_t7", "op": "swiglu", "M": 7, "N": 1408, "dt": "f16"},
        # a prompt between the two products of an MLP
        {"name": "swiglu_t2048", "op": "swiglu", "M": 2048, "N": 11008, "dt": "bf16"},
        # a small linear at one token: latency alone
        {"name": "mm_256x512_b1", "op": "matmul", "M": 256, "N": 512, "b": 1, "dt": "f32", "y": "f32"},
        # a batch of decode tokens through the up projection of an MLP
        {"name": "mm_up_b16", "op": "matmul", "M": 11008, "N": 4096, "b": 16, "dt": "bf16", "y": "bf16"},
        # a short prompt, nothing a multiple of anything
        {"name": "mm_odd_b77", "op": "matmul", "M": 4099, "N": 5003, "b": 77, "dt": "f16", "y": "f16"},
        # the benchmark's prefill product
        {"name": "mm_mlp_70b_prefill", "op": "matmul", "M": 28672, "N": 8192, "b": 2048, "dt": "bf16", "y": "bf16"},
        # one decode token through gate and up (side by side) of the two large experts that it chose
        {"name": "grp_large_t1", "op": "group", "E": 8, "M": 22016, "N": 4096, "T": 1, "k": 2, "tail": 0,
         "rows": False, "dt": "bf16", "y": "bf16"},
        # a small decode batch through gate and up of many small experts
        {"name": "grp_fine_t7", "op": "group", "E": 64, "M": 2816, "N": 2048, "T": 7, "k": 6, "tail": 0,
         "rows": False, "dt": "f16", "y": "f16"},
        # a padded prompt through the down projection of many small experts, its rows encoded by the step before
        {"name": "grp_fine_t500", "op": "group", "E": 64, "M": 2048, "N": 1408, "T": 500, "k": 6, "tail": 72,
         "rows": True, "dt": "f32", "y": "f32"},
        # a prompt through gate and up of large experts
        {"name": "grp_large_t2048", "op": "group", "E": 8, "M": 22016, "N": 4096, "T": 2048, "k": 2, "tail": 0,
         "rows": False, "dt": "bf16", "y": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["encode", "swiglu", "matmul", "matmul", "group", "group"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "encode":
        return {"op": op, "M": _log(rng, 1, 28672), "N": _log(rng, 64, 8192), "dt": dt, "w": rng.random() < 0.5}
    if op == "swiglu":
        return {"op": op, "M": _log(rng, 1, 2048), "N": _log(rng, 64, 11008), "dt": dt}
    if op == "matmul":
        return {"op": op, "M": _log(rng, 64, 28672), "N": _log(rng, 64, 8192), "b": _log(rng, 1, 2048), "dt": dt,
                "y": rng.choice(["f32", dt])}
    E = rng.choice([4, 8, 8, 16, 32, 64, 128])
    N = _log(rng, 256, 4096)
    M = min(_log(rng, 128, 22016), 8 * 22016 * 4096 // (E * N))
    k = rng.randint(1, min(E, 8))
    T = min(_log(rng, 1, 2048), max(1, 4096 * 22016 * 4096 // (k * M * N)))
    return {"op": op, "E": E, "M": M, "N": N, "T": T, "k": k, "tail": rng.choice([0, 0, 1, 37]),
            "rows": rng.random() < 0.4, "dt": dt, "y": rng.choice(["f32", dt])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _weight(shape, std, g, dt):
    """Normal weights whose output rows differ in size."""
    w = torch.randn(shape, generator=g, device=g.device)
    size = torch.rand(shape[:-1] + (1,), generator=g, device=g.device).mul_(1.5).add_(0.25)
    return w.mul_(size * std).to(DT[dt])


def _acts(T, N, g, dt):
    """Normal activations with a few large channels."""
    x = torch.randn((T, N), generator=g, device=g.device)
    big = torch.rand((N,), generator=g, device=g.device) < 0.005
    return torch.where(big, x * 20.0, x).to(DT[dt])


def _routes(T, k, E, g):
    """Experts of T tokens, some more popular than others: (counts [E], the token of each term), int32."""
    logits = torch.randn((T, E), generator=g, device=g.device)
    logits += 0.7 * torch.randn((E,), generator=g, device=g.device)
    ids = torch.topk(logits, k, dim=1).indices.flatten()
    counts = (ids[:, None] == torch.arange(E, device=g.device)).sum(0)
    return counts.to(torch.int32), (torch.sort(ids, stable=True).indices // k).to(torch.int32)


def _data(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    op, M, N = case["op"], case["M"], case["N"]
    if op == "encode":
        return {"x": _weight((M, N), 0.02, g, case["dt"]) if case["w"] else _acts(M, N, g, case["dt"])}
    if op == "swiglu":   # halves of one product's rows
        return {"gu": (1.5 * torch.randn((M, 2 * N), generator=g, device=dev)).to(DT[case["dt"]])}
    if op == "matmul":
        return {"w": _encode(_weight((M, N), 1.0 / math.sqrt(N), g, "bf16")), "x": _acts(case["b"], N, g, case["dt"])}
    T, k, E = case["T"], case["k"], case["E"]
    parts = [_encode(_weight((M, N), 1.0 / math.sqrt(N), g, "bf16")) for _ in range(E)]
    d = {"w": (torch.stack([q for q, _ in parts]), torch.stack([s for _, s in parts]))}
    d["counts"], d["index"] = _routes(T, k, E, g)
    terms = T * k + case["tail"]
    if case["rows"]:
        d["x"] = _encode(_acts(terms, N, g, case["dt"]))
        del d["index"]
    else:
        d["x"] = _acts(T, N, g, case["dt"])
        d["index"] = torch.cat([d["index"], torch.zeros(case["tail"], dtype=torch.int32, device=dev)])
    d["out"] = torch.randn((terms, M), generator=g, device=dev).to(DT[case["y"]])
    return d


def prepare(case, seed):
    st = dict(case, **_data(case, seed))
    if own:
        import sub_bit_weight_sketch_amd as sk
        if "w" in st and case["op"] != "encode":
            st["w"] = sk.int8_tables(*st["w"])
        if case["op"] == "group" and case["rows"]:
            st["x"] = sk.int8_tables(*st["x"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _encode(x):
    """(codes [M, N] int8, scales [M] float32) of x, by rows."""
    v = x.to(torch.float64)
    amax = v.abs().amax(1, keepdim=True)
    codes = torch.round(v * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax))).to(torch.int8)
    return codes, (amax[:, 0] / 127.0).to(torch.float32)


def _product(qx, sx, qw, sw):
    return (qx @ qw.to(torch.float32).t()) * sx[:, None] * sw


def run(st):
    op = st["op"]
    if own:
        import sub_bit_weight_sketch_amd as sk
        if op == "encode":
            t = sk.int8_encode(st["x"], check=False)
            return t.codes(), t.scales()
        if op == "swiglu":
            t = sk.int8_swiglu(st["gu"][:, :st["N"]], st["gu"][:, st["N"]:])
            return t.codes(), t.scales()
        if op == "matmul":
            return sk.int8_matmul(st["w"], st["x"], dtype=DT[st["y"]])
        return sk.int8_matmul_group(st["w"], st["x"], st["counts"], rows=st.get("index"), out=st["out"])
    if op == "encode":
        return _encode(st["x"])
    if op == "swiglu":
        g, u = st["gu"].to(torch.float64).split(st["N"], 1)
        return _encode(g / (1.0 + torch.exp(-g)) * u)
    qx, sx = st["x"] if op == "group" and st["rows"] else _encode(st["x"])
    qx = qx.to(torch.float32)
    if op == "matmul":
        return _product(qx, sx, *st["w"]).to(DT[st["y"]])
    sizes = st["counts"].tolist()
    if not st["rows"]:
        qx, sx = qx[st["index"]], sx[st["index"]]
    end = 0
    for e, n in enumerate(sizes):
        if n:
            at, end = end, end + n
            st["out"][at:end] = _product(qx[at:end], sx[at:end], st["w"][0][e], st["w"][1][e])
    return st["out"]


def work(case):
    op, M, N, es = case["op"], case["M"], case["N"], ES[case["dt"]]
    if op == "encode":
        return {"bytes": M * N * (es + 1) + 4 * M, "flops": 2 * M * N}
    if op == "swiglu":
        return {"bytes": M * N * (2 * es + 1) + 4 * M, "flops": 8 * M * N}
    if op == "matmul":
        b = case["b"]
        return {"bytes": M * (N + 4) + b * N * es + b * M * ES[case["y"]], "flops": 2 * b * M * N}
    T, k, E = case["T"], case["k"], case["E"]
    active = E * (1.0 - (1.0 - k / E) ** T)            # experts some token takes, routed evenly
    terms = T * k
    x = terms * (N + 4) if case["rows"] else T * N * es + 4 * terms
    return {"bytes": int(active * M * (N + 4)) + x + 4 * E + terms * M * ES[case["y"]], "flops": 2 * terms * M * N}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _definition(v):
    """(codes, scales) of rows of float64: twice the code's size, rounded down,
    decides between the two integers beside it; an exact half goes to the even one."""
    big = v.abs().max(1).values
    twice = 254.0 * v.abs()
    per = torch.where(big > 0, big, torch.ones_like(big))[:, None]
    n = torch.floor(twice / per)
    low = torch.floor(n / 2)
    half = (n == 2 * low + 1) & (twice == n * per)
    up = (n == 2 * low + 1) & ~(half & (low % 2 == 0))
    return torch.where(v < 0, -1.0, 1.0) * (low + up.double()), (big / 127.0).float().double()


def exact(case, seed):
    d = _data(case, seed)
    if case["op"] == "encode":
        q, s = _definition(d["x"].double())
        return q.to(torch.int8), s
    if case["op"] == "swiglu":
        gate, up = d["gu"][:, :case["N"]].double(), d["gu"][:, case["N"]:].double()
        q, s = _definition(gate * torch.sigmoid(gate) * up)
        return q.to(torch.int8), s
    if case["op"] == "matmul":
        q, s = _definition(d["x"].double())
        return torch.outer(s, d["w"][1].double()) * torch.matmul(q, d["w"][0].double().t())
    q, s = (d["x"][0].double(), d["x"][1].double()) if case["rows"] else _definition(d["x"].double())
    y = d["out"].double()
    i = 0
    for e in range(case["E"]):
        take = torch.arange(i, i + int(d["counts"][e]), device=y.device)
        i += take.numel()
        if take.numel():
            r = take if case["rows"] else d["index"][take].long()
            y[take] = torch.matmul(q[r] * s[r, None], d["w"][0][e].double().t()) * d["w"][1][e].double()
    return y
