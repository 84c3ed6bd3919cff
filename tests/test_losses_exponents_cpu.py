"""The exponents of the losses' kernels in float32, step by step on the CPU: formed
from the rounded product m c up to |m c| = 2^20, from z - m above, and joined where
one part of a row is formed in one way and one in the other.  Each is off by a few
units (2^-24) of its distance from the largest, and all of a row by the rounding of
m c, 2^-5 at most, which drops out."""
import numpy as np

F = np.float32
LOG2E = F(1.4426950408889634)
U = 2.0 ** -24


def product(x, c):
    return np.float64(x) * np.float64(c)  # exact: 48 bits


def fused(m, c):
    with np.errstate(over="ignore"):
        return bool(np.abs(m * c) <= F(2.0 ** 20))


def rounded(m, c):
    return np.float64(m * c) if fused(m, c) else product(m, c)


def exponent(z, m, c):
    if fused(m, c):
        return F(product(z, c) - np.float64(m * c))
    return (z - m) * c


def factor(m, old, c):
    """The exponent of what takes exponentials compared with `old` to those compared with m."""
    if fused(m, c) and fused(old, c):
        return old * c - m * c
    if not fused(m, c) and not fused(old, c):
        return (old - m) * c
    return F(rounded(old, c) - rounded(m, c))


def test_exponents_of_any_logits():
    g = np.random.default_rng(1)
    seen = set()
    for power in range(128):
        for _ in range(60):
            c = LOG2E / F(2.0 ** g.integers(-60, 61)) if g.random() < 0.7 else LOG2E
            size = min(power - np.log2(np.float64(c)) + g.random() - 1, 127)
            m = F(np.exp2(size) * g.choice((-1, 1)))
            below = np.exp2(g.uniform(-25, 1)) * np.abs(np.float64(m))
            if g.random() < 0.3:
                below = np.exp2(g.uniform(-5, 5)) / np.float64(c)
            old = F(max(np.float64(m) - below, -3.4e38))
            z = F(max(np.float64(old) - below * g.random(), -3.4e38))
            with np.errstate(over="ignore"):
                x = np.float64(exponent(z, old, c)) + np.float64(factor(m, old, c))
                own = np.float64(exponent(m, m, c))
            far = (np.float64(m) - np.float64(z)) * np.float64(c)
            if far > 2.0 ** 127:  # float32 has no such number: infinite, a weight of 0
                continue
            assert abs(own) <= 2.0 ** -5
            assert abs(x + far - own) <= 5 * U * (far + 1), (power, m, old, z, c)
            seen.add((fused(m, c), fused(old, c)))
    assert len(seen) == 4


def test_the_rounding_alone_would_not_do():
    """What the limit is for: |m c| = 2^31 has a rounding of up to 128, the exponent of
    the largest term."""
    m = F(-1e10)
    assert abs(product(m, LOG2E) - np.float64(m * LOG2E)) > 200
    assert exponent(m, m, LOG2E) == 0 and not fused(m, LOG2E)
