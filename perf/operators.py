"""Operators on 8-bit floating-point weights: what they compute and how they are timed.

Three operators, on matrices held as e4m3 codes with one power-of-two scale
(e8m0) for each block of 128 columns:

  encode  W [M, N] -> codes [M, N] (e4m3) and scales: one for each block of
          128 x 128 (weights) or of 1 x 128 (activations, row by row)
  matmul  Y = X8 . W8^T, W8 an encoded weight, X8 the rows of X encoded by
          blocks of 1 x 128 on the way in; Y float32, bfloat16 or binary16
  moe     a mixture-of-experts layer for a few tokens: router, softmax, the
          top k of E experts, SwiGLU experts on encoded weights, their
          weighted sum; Y float32, the chosen experts and their weights

The scale of a block is 2^e with the smallest e >= -127 such that the block's
largest magnitude is at most 448 * 2^e; a code is the e4m3 value next to
x / 2^e, ties to even.  The last block of a row covers what is left of it.

With ``own`` false, ``run`` computes in elementary torch operations; with
``own`` true it calls the library.
"""
import math

import torch

own = False

B = 128                      # columns of a block
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ES = {"f32": 4, "bf16": 2, "f16": 2}


def _ceil(a, b):
    return -(-a // b)


def listed():
    return [
        # the largest linear of the benchmark, encoded once while a model is loaded, beyond the last-level cache
        {"name": "encode_w_mlp_70b", "op": "encode", "M": 28672, "N": 8192, "rows": 128, "dt": "bf16"},
        # activations of a prompt, row by row, an odd number of tokens and of columns
        {"name": "encode_rows_odd", "op": "encode", "M": 517, "N": 4001, "rows": 1, "dt": "f32"},
        # a small linear at one token: latency alone
        {"name": "mm_256x512_b1", "op": "matmul", "M": 256, "N": 512, "b": 1, "dt": "f32", "y": "f32"},
        # one decode step of an attention projection
        {"name": "mm_attn_b1", "op": "matmul", "M": 4096, "N": 4096, "b": 1, "dt": "bf16", "y": "bf16"},
        # a batch of decode tokens through the up projection of an MLP
        {"name": "mm_up_b16", "op": "matmul", "M": 11008, "N": 4096, "b": 16, "dt": "bf16", "y": "bf16"},
        # a short prompt, nothing a multiple of anything
        {"name": "mm_odd_b77", "op": "matmul", "M": 4099, "N": 5003, "b": 77, "dt": "f16", "y": "f16"},
        # a prompt through the up projection, summed and returned in float32
        {"name": "mm_up_b512_f32", "op": "matmul", "M": 11008, "N": 4096, "b": 512, "dt": "bf16", "y": "f32"},
        # the benchmark's prefill product
        {"name": "mm_mlp_70b_prefill", "op": "matmul", "M": 28672, "N": 8192, "b": 2048, "dt": "bf16", "y": "bf16"},
        # a toy layer at one token: latency alone
        {"name": "moe_small_t1", "op": "moe", "H": 512, "I": 256, "E": 8, "k": 2, "T": 1, "norm": True, "dt": "f32"},
        # one decode token through a layer of large experts
        {"name": "moe_large_t1", "op": "moe", "H": 4096, "I": 11008, "E": 8, "k": 2, "T": 1, "norm": True,
         "dt": "bf16"},
        # a decode batch: every large expert has a few tokens
        {"name": "moe_large_t16", "op": "moe", "H": 4096, "I": 11008, "E": 8, "k": 2, "T": 16, "norm": True,
         "dt": "bf16"},
        # many small experts, softmax weights as they are, an odd batch
        {"name": "moe_fine_t7", "op": "moe", "H": 2048, "I": 1408, "E": 64, "k": 6, "T": 7, "norm": False, "dt": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["encode", "matmul", "matmul", "moe", "moe"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "encode":
        return {"op": op, "M": _log(rng, 1, 28672), "N": _log(rng, 64, 8192), "rows": rng.choice([1, 128]), "dt": dt}
    if op == "matmul":
        return {"op": op, "M": _log(rng, 64, 28672), "N": _log(rng, 64, 8192), "b": _log(rng, 1, 2048), "dt": dt,
                "y": rng.choice(["f32", dt])}
    E = rng.choice([4, 8, 8, 16, 32, 64, 128])
    H = _log(rng, 256, 4096)
    I = min(_log(rng, 128, 11008), 8 * 4096 * 11008 // (E * H))
    return {"op": op, "H": H, "I": I, "E": E, "k": rng.randint(1, min(E, 8)), "T": _log(rng, 1, 32),
            "norm": rng.random() < 0.5, "dt": dt}


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


def _data(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    if case["op"] == "encode":
        f = _weight if case["rows"] == 128 else None
        return {"x": f((case["M"], case["N"]), 0.02, g, case["dt"]) if f else _acts(case["M"], case["N"], g, case["dt"])}
    if case["op"] == "matmul":
        M, N = case["M"], case["N"]
        return {"w": _encode(_weight((M, N), 1.0 / math.sqrt(N), g, "bf16"), 128),
                "x": _acts(case["b"], N, g, case["dt"])}
    H, I, E = case["H"], case["I"], case["E"]
    d = {"router": _weight((E, H), 1.0 / math.sqrt(H), g, case["dt"]), "x": _acts(case["T"], H, g, case["dt"])}
    for name, M, N in (("gate", I, H), ("up", I, H), ("down", H, I)):
        parts = [_encode(_weight((M, N), 1.0 / math.sqrt(N), g, "bf16"), 128) for _ in range(E)]
        d[name] = (torch.stack([c.view(torch.uint8) for c, _ in parts]).view(torch.float8_e4m3fn),
                   torch.stack([s for _, s in parts]))
    return d


def prepare(case, seed):
    d = _data(case, seed)
    st = dict(case, **d)
    if own:
        import sub_bit_weight_sketch_amd as sk
        if case["op"] == "matmul":
            st["w"] = sk.fp8_tables(*d["w"])
        elif case["op"] == "moe":
            st["layer"] = sk.MoE(d["router"], sk.fp8_tables(*d["gate"]), sk.fp8_tables(*d["up"]),
                                 sk.fp8_tables(*d["down"]), case["k"], renorm=case["norm"])
            for name in ("gate", "up", "down"):
                del st[name]
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _blocks(x, rows):
    """x padded with zeros to whole blocks, as [row blocks, rows, column blocks, 128] float32."""
    M, N = x.shape
    p = torch.zeros((_ceil(M, rows) * rows, _ceil(N, B) * B), dtype=torch.float32, device=x.device)
    p[:M, :N] = x
    return p.view(-1, rows, _ceil(N, B), B)


def _encode(x, rows):
    """(codes [M, N] float8_e4m3fn, biased exponents [row blocks, column blocks] uint8)"""
    M, N = x.shape
    v = _blocks(x, rows)
    amax = v.abs().amax(dim=(1, 3))
    bits = amax.view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(min=0)
    inv = torch.exp2((127 - byte).to(torch.float32))
    codes = (v * inv[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(v.shape[0] * rows, -1)[:M, :N].contiguous(), byte.to(torch.uint8)


def _decode(codes, scales, rows):
    M, N = codes.shape
    s = torch.exp2(scales.to(torch.float32) - 127.0)
    s = s.repeat_interleave(rows, 0)[:M].repeat_interleave(B, 1)[:, :N]
    return codes.to(torch.float32) * s


def _moe(st):
    k, E = st["k"], st["E"]
    logits = st["x"].double() @ st["router"].double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :k], order.values[:, :k]
    w = torch.exp(top - top[:, :1])
    total = w.sum(1, keepdim=True) if st["norm"] else torch.exp(logits - top[:, :1]).sum(1, keepdim=True)
    w = (w / total).to(torch.float32)
    x = st["x"].to(torch.float32)
    y = torch.zeros((st["T"], st["H"]), dtype=torch.float32, device=x.device)
    for e in range(E):
        we = torch.where(ids == e, w, torch.zeros_like(w)).sum(1, keepdim=True)
        gate, up, down = (_decode(st[n][0][e], st[n][1][e], 128) for n in ("gate", "up", "down"))
        g, u = x @ gate.t(), x @ up.t()
        y += we * (((g / (1.0 + torch.exp(-g))) * u) @ down.t())
    return y, ids.to(torch.int32), w


def run(st):
    op = st["op"]
    if own:
        import sub_bit_weight_sketch_amd as sk
        if op == "encode":
            t = sk.fp8_encode(st["x"], block_rows=st["rows"], check=False)
            return t.codes(), t.scales()
        if op == "matmul":
            return sk.fp8_matmul(st["w"], st["x"], dtype=DT[st["y"]])
        return sk.moe(st["layer"], st["x"], return_routing=True)
    if op == "encode":
        return _encode(st["x"], st["rows"])
    if op == "matmul":
        x = _decode(*_encode(st["x"], 1), 1)
        return (x @ _decode(*st["w"], 128).t()).to(DT[st["y"]])
    return _moe(st)


def work(case):
    if case["op"] == "encode":
        M, N = case["M"], case["N"]
        scales = _ceil(M, case["rows"]) * _ceil(N, B)
        return {"bytes": M * N * (ES[case["dt"]] + 1) + scales, "flops": 2 * M * N}
    if case["op"] == "matmul":
        M, N, b = case["M"], case["N"], case["b"]
        w = M * N + _ceil(M, B) * _ceil(N, B)
        return {"bytes": w + b * N * ES[case["dt"]] + b * M * ES[case["y"]], "flops": 2 * b * M * N}
    H, I, E, k, T = (case[n] for n in ("H", "I", "E", "k", "T"))
    active = E * (1.0 - (1.0 - k / E) ** T)            # experts some token takes, routed evenly
    expert = 3 * H * I + 2 * _ceil(I, B) * _ceil(H, B) + _ceil(H, B) * _ceil(I, B)
    io = (E + T) * H * ES[case["dt"]] + T * (4 * H + 8 * k)
    return {"bytes": int(active * expert) + io, "flops": 2 * T * (E * H + 3 * k * H * I)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(v):
    """float64 -> the nearest e4m3 value (3 mantissa bits, least exponent -6), ties to even."""
    _, e = torch.frexp(v)
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.round(v / step) * step


def _definition(x, rows):
    """(values of the codes in float64, exponents) straight from the definition."""
    M, N = x.shape
    out = torch.empty((M, N), dtype=torch.float64, device=x.device)
    exps = torch.empty((_ceil(M, rows), _ceil(N, B)), dtype=torch.int64, device=x.device)
    for c in range(exps.shape[1]):
        v = x[:, c * B:(c + 1) * B].double()
        big = v.abs().amax(1)
        if rows > 1:
            pad = torch.zeros(exps.shape[0] * rows, dtype=torch.float64, device=x.device)
            pad[:M] = big
            big = pad.view(-1, rows).amax(1)
        m, e = torch.frexp(big / 448.0)                # big / 448 = m 2^e, 0.5 <= m < 1
        e = torch.where(m == 0.5, e - 1, e).clamp(min=-127)
        e = torch.where(big == 0, torch.full_like(e, -127), e)
        s = torch.exp2(e.double())
        exps[:, c] = e
        out[:, c * B:(c + 1) * B] = _e4m3(v / s.repeat_interleave(rows)[:M, None])
    return out, exps


def _value(codes, exps, rows):
    full = torch.exp2(exps.double()).repeat_interleave(rows, 0)[:codes.shape[0]]
    v = codes.double()
    for c in range(full.shape[1]):
        v[:, c * B:(c + 1) * B] *= full[:, c:c + 1]
    return v


def exact(case, seed):
    d = _data(case, seed)
    if case["op"] == "encode":
        v, e = _definition(d["x"], case["rows"])
        return v, (e + 127).to(torch.uint8)
    if case["op"] == "matmul":
        x = _value(*_definition(d["x"], 1), 1)
        return x @ _value(d["w"][0], d["w"][1].long() - 127, 128).t()
    T, H, k = case["T"], case["H"], case["k"]
    x = d["x"].double()
    logits = x @ d["router"].double().t()
    p = torch.softmax(logits, dim=1)
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    chosen, weights = [], []
    for t in range(T):
        row = logits[t].tolist()
        best = sorted(range(case["E"]), key=lambda e: (-row[e], e))[:k]
        chosen.append(best)
        weights.append(torch.stack([p[t, e] for e in best]))
    w = torch.stack(weights)
    if case["norm"]:
        w = w / w.sum(1, keepdim=True)
    for e in sorted({e for best in chosen for e in best}):
        gate, up, down = (_value(d[n][0][e], d[n][1][e].long() - 127, 128) for n in ("gate", "up", "down"))
        for t in range(T):
            if e in chosen[t]:
                g = gate @ x[t]
                h = g * torch.sigmoid(g) * (up @ x[t])
                y[t] += w[t, chosen[t].index(e)] * (down @ h)
    return y, torch.tensor(chosen, dtype=torch.int32, device=x.device), w
