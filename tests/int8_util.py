"""Plain forms of the 8-bit integer operators for the tests (NumPy, CPU),
written from the definitions in include/sketch_int8.h."""
import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def randn(shape, seed, scale=1.0, dt="f32"):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(DT[dt])


def to64(t):
    """Device or host tensor -> float64 array (exact)."""
    return t.detach().cpu().to(torch.float64).numpy()


def encode(x):
    """(codes [M, N] int64, scales [M] float32) of float64 values that float32
    holds.  n = floor(254 |x| / amax) is settled by exact products (8 bits of n
    times 24 of amax); a code is n / 2 rounded up where n is odd, but for an exact
    half beside an even integer."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    amax = np.abs(np.where(bad[:, None], 0.0, x)).max(axis=1, initial=0.0)
    per = np.where(amax > 0, amax, 1.0)[:, None]
    twice = 254.0 * np.abs(np.where(bad[:, None], 0.0, x))
    n = np.floor(twice / per)
    n -= n * per > twice
    n += (n + 1) * per <= twice
    low = np.floor(n / 2)
    odd = n % 2 == 1
    even_half = odd & (n * per == twice) & (low % 2 == 0)
    code = np.where(odd & ~even_half, low + 1, low)
    code = np.where(x < 0, -code, code).astype(np.int64)
    with np.errstate(under="ignore"):
        scale = (amax / 127.0).astype(np.float32)
    return np.where(bad[:, None], 0, code), np.where(bad, np.float32("nan"), scale).astype(np.float32)


def swiglu(g, u):
    """silu(g) * u in extended precision."""
    g, u = np.asarray(g, dtype=np.longdouble), np.asarray(u, dtype=np.longdouble)
    with np.errstate(all="ignore"):
        return g / (1 + np.exp(-g)) * u


def product(qx, sx, qw, sw, dt):
    """The product's bits: exact sums (below 2^31, float64 holds them), one
    rounding to float32, one for each scale, one to the type of Y."""
    total = qx.astype(np.float64) @ qw.astype(np.float64).T
    with np.errstate(all="ignore"):
        y = total.astype(np.float32) * sx.astype(np.float32)[:, None] * sw.astype(np.float32)[None, :]
    return torch.from_numpy(np.ascontiguousarray(y)).to(DT[dt])


def table(t):
    """(codes int64, scales float32) of an Int8Tables."""
    return t.codes().cpu().numpy().astype(np.int64), t.scales().cpu().numpy()


def same(got, want):
    """Equal bit for bit, NaN as NaN."""
    got = got.detach().cpu()
    assert got.shape == want.shape and got.dtype == want.dtype
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    zero = torch.zeros((), dtype=want.dtype)
    a, b = torch.where(nan, zero, got), torch.where(nan, zero, want)
    if not torch.equal(a, b):
        bad = (a != b).nonzero()
        raise AssertionError("%d of %d differ, first at %s: %r, want %r" % (
            len(bad), want.numel(), bad[0].tolist(), a[tuple(bad[0])].item(), b[tuple(bad[0])].item()))


def spans(counts, terms):
    """(expert, first, end) of the experts that have terms, by the rules of the counts."""
    at, out = 0, []
    for e, c in enumerate(np.asarray(counts).tolist()):
        end = min(at + max(c, 0), terms)
        if end > at:
            out.append((e, at, end))
        at = end
    return out


def group(qx, sx, rows, counts, qw, sw, out):
    """The grouped product on a copy of `out`; a row outside X gives NaN."""
    out = out.clone()
    dt = next(k for k, v in DT.items() if v == out.dtype)
    for e, at, end in spans(counts, out.shape[0]):
        r = np.arange(at, end) if rows is None else np.asarray(rows)[at:end]
        ok = (r >= 0) & (r < qx.shape[0])
        rr = np.where(ok, r, 0)
        out[at:end] = product(qx[rr], np.where(ok, sx[rr], np.float32("nan")), qw[e], sw[e], dt)
    return out


def ragged(E, terms, seed, empty=0.3):
    """Counts of E experts that add up to `terms`, some of them zero."""
    g = np.random.default_rng(seed)
    p = g.gamma(0.7, size=E) * (g.random(E) >= empty) + 1e-9
    return g.multinomial(terms, p / p.sum()).tolist()
