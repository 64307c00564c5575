"""Plain 64-bit forms of the e4m3 operators for the tests (NumPy, CPU),
written from the definitions in include/sketch_fp8.h."""
import numpy as np
import torch

EPS32 = 2.0 ** -24      # half a step of float32, relative


def blocks(n, b):
    return -(-n // b)


def e4m3_round(v):
    """float64 -> the nearest e4m3 value (3 mantissa bits, least exponent -6), ties to even."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 1, -6).astype(np.float64) - 3)
    return np.rint(v / step) * step


def e4m3_value(bits):
    """uint8 codes -> float64 values, by the fields of the format."""
    bits = np.asarray(bits, dtype=np.uint8).astype(np.int64)
    sign = np.where(bits & 0x80, -1.0, 1.0)
    ex, man = (bits >> 3) & 15, bits & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (1.0 + man / 8.0) * np.exp2((ex - 7).astype(np.float64)))
    return np.where((bits & 0x7F) == 0x7F, np.nan, sign * v)


def encode(x, rows):
    """(values of the codes [M, N] float64, biased exponents [row blocks, column blocks])"""
    x = np.asarray(x, dtype=np.float64)
    M, N = x.shape
    out = np.zeros((M, N))
    byte = np.zeros((blocks(M, rows), blocks(N, 128)), dtype=np.int64)
    for i in range(byte.shape[0]):
        for j in range(byte.shape[1]):
            b = x[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
            if not np.isfinite(b).all():
                byte[i, j] = 255
                out[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128] = np.nan
                continue
            amax, e = np.abs(b).max(), -127
            while amax > 448.0 * 2.0 ** e:
                e += 1
            byte[i, j] = e + 127
            out[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128] = e4m3_round(b / 2.0 ** e)
    return out, byte


def values(codes, byte, rows):
    """The numbers that codes (values) and exponents stand for."""
    M, N = codes.shape
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127.0))
    return codes * s.repeat(rows, 0)[:M].repeat(128, 1)[:, :N]


def encoded(x, rows):
    return values(*encode(x, rows), rows)


def to64(t):
    """Device or host tensor -> float64 array (exact)."""
    return t.detach().cpu().to(torch.float64).numpy()


def table_values(t):
    """The numbers of an Fp8Tables, decoded here from its codes and scale bytes."""
    c = e4m3_value(t.codes().view(torch.uint8).cpu().numpy())
    s = t.scales().cpu().numpy()
    if t.count is None:
        return values(c, s.astype(np.int64), t.block_rows)
    return np.stack([values(c[i], s[i].astype(np.int64), t.block_rows) for i in range(t.count)])


def moe(x, router, gate, up, down, k, renorm):
    """(y, ids, weights) in float64; NaN logits rank first, ties go to the lower expert."""
    T, E = x.shape[0], router.shape[0]
    with np.errstate(all="ignore"):
        logits = x @ router.T
        ids = np.zeros((T, k), dtype=np.int64)
        w = np.zeros((T, k))
        y = np.zeros((T, down.shape[1]))
        for t in range(T):
            rank = [(0, 0.0, e) if np.isnan(v) else (1, -v, e) for e, v in enumerate(logits[t])]
            ids[t] = [r[2] for r in sorted(rank)[:k]]
            top = logits[t, ids[t]]
            ex = np.exp(top - top[0])
            w[t] = ex / (ex.sum() if renorm else np.exp(logits[t] - top[0]).sum())
            for s, e in enumerate(ids[t]):
                g, u = gate[e] @ x[t], up[e] @ x[t]
                y[t] += w[t, s] * (down[e] @ (g / (1.0 + np.exp(-g)) * u))
    return y, ids, w
