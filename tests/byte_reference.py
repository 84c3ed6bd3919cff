"""Plain reference of the rows in 8 bits in float64 (numpy), for the tests."""
import numpy as np


def grid():
    """The values of the 127 codes without sign, in order."""
    c = np.arange(127)
    power, part = c >> 3, c & 7
    return np.where(power > 0, (1 + part / 8) * np.exp2(power - 7.0), part / 512)


GRID = grid()


def groups(dim):
    return -(-dim // 128)


def scale_bytes(dim):
    return 4 * -(-groups(dim) // 4)


def quantize(x):
    """(codes, scales) of rows, by the definition: the nearest grid value, a
    midpoint to the even code."""
    x = np.asarray(x, dtype=np.float64)
    n, dim = x.shape
    g = groups(dim)
    b = np.zeros((n, 128 * g))
    b[:, :dim] = x
    b = b.reshape(n, g, 128)
    neg = np.signbit(b)
    bad = ~np.isfinite(b).all(2)
    b = np.abs(np.where(bad[:, :, None], 0, b))
    top = b.max(2)
    part, e = np.frexp(top)  # top = part 2^e, 1/2 <= part < 1; 448 = 0.875 * 2^9
    e = np.where(top > 0, np.maximum(e - 9 + (part > 0.875), -127), -127)
    v = b / np.exp2(e.astype(np.float64))[:, :, None]
    assert v.max(initial=0) <= 448
    mid = (GRID[1:] + GRID[:-1]) / 2
    down, up = np.searchsorted(mid, v, side="left"), np.searchsorted(mid, v, side="right")
    code = np.where(down % 2 == 0, down, up) + 128 * neg
    code = np.where(bad[:, :, None], 0, code).reshape(n, -1).astype(np.uint8)
    scales = np.zeros((n, scale_bytes(dim)), np.uint8)
    scales[:, :g] = np.where(bad, 255, e + 127)
    return code, scales


def values(codes, scales, dim):
    """The float64 values that 8-bit rows stand for."""
    v = np.where(codes & 128, -1.0, 1.0) * np.append(GRID, np.nan)[codes & 127]
    s = np.exp2(scales.astype(np.float64) - 127)
    s = np.where(scales == 255, np.nan, s)[:, :codes.shape[1] // 128].repeat(128, axis=1)
    return (v * s)[:, :dim]
