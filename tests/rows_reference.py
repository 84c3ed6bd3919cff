"""Plain references of the row operators in float64 (numpy), for the tests."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def groups(dim):
    return -(-dim // 128)


def quantize(x):
    """(codes, scales) of rows, by the definition: the nearest grid value, a
    midpoint to the even code, magnitudes above the grid to its largest."""
    x = np.asarray(x, dtype=np.float64)
    n, dim = x.shape
    b = np.zeros((n, 128 * groups(dim)))
    b[:, :dim] = x
    neg = np.signbit(b).reshape(n, -1, 32)
    b = b.reshape(n, -1, 32)
    bad = ~np.isfinite(b).all(2)
    top = np.where(np.isfinite(b), np.abs(b), 0).max(2)
    # frexp: top = m 2^e with 1/2 <= m < 1, so floor(log2 top) = e - 1
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127).clip(-127, None)
    v = np.abs(np.where(np.isfinite(b), b, 0)) / np.exp2(e.astype(np.float64))[:, :, None]
    mid = (GRID[1:] + GRID[:-1]) / 2
    down, up = np.searchsorted(mid, v, side="left"), np.searchsorted(mid, v, side="right")
    code = np.where(down % 2 == 0, down, up) + 8 * neg
    code = np.where(bad[:, :, None], 0, code).reshape(n, -1).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def values(codes, scales, dim):
    """The float64 values that 4-bit rows stand for."""
    n = codes.shape[0]
    c = np.empty((n, 2 * codes.shape[1]), dtype=np.int64)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    s = np.exp2(scales.astype(np.float64) - 127)
    s = np.where(scales == 255, np.nan, s).repeat(32, axis=1)
    return (np.where(c & 8, -1.0, 1.0) * GRID[c & 7] * s)[:, :dim]


def kept(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Weights of one row after the truncations (float64; zero where cut)."""
    z = np.asarray(z, dtype=np.float64) + 0.0
    w = np.where(z > -np.inf, np.exp((z - z.max()) / temperature), 0.0)
    order = np.argsort(-z, kind="stable")
    n = len(z)
    rank = np.empty(n, dtype=np.int64)
    rank[order] = np.arange(n)
    stay = np.ones(n, dtype=bool)
    if 1 <= top_k < n:
        stay &= rank < top_k
    if top_p < 1:
        total = w[stay].sum()
        before = np.concatenate(([0.0], np.cumsum(w[order])[:-1]))[rank]
        stay &= (before < top_p * total) | (rank == 0)
    if min_p > 0:
        stay &= w >= min(min_p, 1.0)
    return np.where(stay, w, 0.0)


def draw(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The component that one row draws; -1 without a distribution."""
    z = np.asarray(z, dtype=np.float64)
    if np.isnan(z).any() or (z == np.inf).any() or not (z > -np.inf).any():
        return -1
    if not temperature > 0:
        return int(np.argmax(z + 0.0))
    w = kept(z, temperature, top_k, top_p, min_p)
    run = np.cumsum(w)
    last = int(np.flatnonzero(w)[-1])
    if not u < 1:
        return last
    return min(int(np.searchsorted(run, max(float(u), 0.0) * run[-1], side="right")), last)
