"""Rows in 8 bits on the GPU against the float64 reference.

Quantisation and its inverse are exact: codes, scales and values have to be
equal.  Products: every term is exact in float32; a sum of D terms in any order,
each addition off by at most 2^-23 of its result (whether the matrix unit rounds
or truncates), is off by at most D 2^-23 sum |a b|; the bias adds one rounding
and the result type one of eps / 2.  With 16-bit results each of 8 neighbouring
terms may be cut at 2^-13 of the largest of them: 8 2^-13 of that largest for
the 8.  Operands of float32 results are held in bfloat16, whose last bit is
2^-133: a value below 2^-130 (4 significant bits) is off by up to 2^-134."""
import numpy as np
import pytest
import torch

import soft_clustering_amd as sc
from tests import byte_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- quantisation

@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 128), (3, 31), (5, 129), (64, 128), (17, 487), (33, 1000), (2, 8192),
                                      (257, 513), (1, 640), (1000, 7)])
def test_quantize_and_back(rows, dim, dtype):
    g = gen(rows * 10007 + dim)
    x = (randn(g, rows, dim) * torch.exp(3 * randn(g, rows, 1))).to(dtype)
    q = sc.byte_quantize(x)
    codes, scales = R.quantize(f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    v = R.values(codes, scales, dim)
    for out in TYPES:
        got = sc.byte_dequantize(q, dtype=out)
        want = torch.from_numpy(v).to(out)
        assert torch.equal(got.cpu(), want)


def test_quantize_every_border():
    """Every grid value and midpoint with its neighbours, and largest values on
    both sides of 448, at scales from the smallest to the largest."""
    mid = (R.GRID[1:] + R.GRID[:-1]) / 2
    base = np.concatenate([R.GRID, mid]).astype(np.float32)
    near = np.concatenate([base, np.nextafter(base, np.float32(500)), np.nextafter(base, np.float32(-500)), -base])
    tops = np.float32([448, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(999)),
                       256, 511, 225])
    rows = []
    for e in (-149, -140, -136, -130, -127, -126, -125, -20, 0, 60, 118, 119):
        for t in tops:
            for part in np.array_split(near[np.abs(near) <= 448], 9):
                r = np.zeros(128)
                r[0] = t
                r[1:1 + len(part)] = part
                with np.errstate(over="ignore"):
                    rows.append(np.ldexp(r, e).astype(np.float32))
    x = np.stack(rows)
    x = x[np.isfinite(x).all(1)]
    q = sc.byte_quantize(torch.from_numpy(x).to(DEV))
    codes, scales = R.quantize(x)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    back = sc.byte_dequantize(q).cpu().numpy()
    want = R.values(codes, scales, 128).astype(np.float32)
    assert np.array_equal(back, want) and np.array_equal(np.signbit(back), np.signbit(want))


def test_dequantize_every_code():
    """Each of the 256 codes (the NaN codes among them) at scales over the range."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (6, 1))
    scales = np.zeros((6, 4), np.uint8)
    scales[:, :2] = [[0, 1], [2, 9], [100, 127], [140, 200], [238, 239], [246, 246]]
    rows = sc.ByteRows(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), 256)
    v = R.values(codes, scales, 256)
    for dtype in TYPES:
        got = sc.byte_dequantize(rows, dtype=dtype).cpu()
        want = torch.from_numpy(v).to(dtype)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(nan=0.5), want.nan_to_num(nan=0.5))


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_quantize_non_finite_blocks(dtype):
    x = randn(gen(1), 6, 300).to(dtype)
    x[1, 5], x[2, 140], x[3, 299], x[4] = float("nan"), float("inf"), float("-inf"), 0
    q = sc.byte_quantize(x)
    codes, scales = R.quantize(f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    back = f64(sc.byte_dequantize(q, dtype=dtype))
    assert np.isnan(back[1, :128]).all() and np.isfinite(back[1, 128:]).all()
    assert np.isnan(back[2, 128:256]).all() and np.isnan(back[3, 256:]).all()
    assert (back[4] == 0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_quantize_strides_and_outputs(dtype):
    """Rows of a wider matrix at an odd offset; codes and scales into a part of
    larger buffers, whose other bytes stay as they are."""
    x = randn(gen(2), 40, 300).to(dtype)[3:30, 7:7 + 201]
    want = sc.byte_quantize(x.contiguous())
    codes = torch.full((40, 320), 171, dtype=torch.uint8, device=DEV)
    scales = torch.full((40, 12), 205, dtype=torch.uint8, device=DEV)
    out = sc.ByteRows(codes[5:32, 16:272], scales[5:32, 4:8], 201)
    sc.byte_quantize(x, out=out)
    assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
    codes[5:32, 16:272], scales[5:32, 4:8] = 171, 205
    assert bool((codes == 171).all()) and bool((scales == 205).all())
    wide = torch.full((27, 210), 3.0, dtype=dtype, device=DEV)
    sc.byte_dequantize(want, dtype=dtype, out=wide[:, 1:202])
    assert torch.equal(wide[:, 1:202], sc.byte_dequantize(want, dtype=dtype))
    assert bool((wide[:, 0] == 3).all()) and bool((wide[:, 202:] == 3).all())


# ---- products

def largest_of_eights(a, b):
    """Sums over groups of 8 neighbouring terms of the largest magnitude among them."""
    total = np.zeros((len(a), len(b)))
    for d in range(0, a.shape[1], 8):
        top = np.zeros_like(total)
        for e in range(d, min(d + 8, a.shape[1])):
            np.maximum(top, np.abs(np.outer(a[:, e], b[:, e])), out=top)
        total += top
    return total


def check_product(A, B, a_val, b_val, dim, bias, dtype):
    got = sc.byte_product(A, B, bias=bias, dtype=dtype)
    assert got.dtype == dtype
    want = a_val @ b_val.T
    mag = np.abs(a_val) @ np.abs(b_val).T
    if bias is not None:
        want, mag = want + f64(bias)[None], mag + np.abs(f64(bias))[None]
    err = np.abs(f64(got) - want)
    eps = torch.finfo(dtype).eps / 2
    tol = (dim + 2) * 2.0 ** -23 * mag + eps * np.abs(want) * 1.001 + torch.finfo(dtype).tiny
    if dtype != torch.float32:
        tol += 2.0 ** -10 * largest_of_eights(a_val, b_val)
    assert np.isfinite(f64(got)).all()
    worst = (err / tol).max() if err.size else 0.0
    assert worst <= 1, f"error {worst:.3g} of the bound"


SIZES = [(1, 16, 128), (1, 1, 1), (1, 1000, 4096), (5, 33, 100), (16, 129, 1000), (17, 50, 1000), (33, 65, 257),
         (64, 200, 768), (65, 31, 128), (128, 128, 128), (129, 257, 640), (300, 500, 1000), (1024, 300, 96),
         (70, 1, 33), (257, 513, 1152), (1, 9000, 300), (40, 9000, 300), (2, 70, 8192), (16, 8300, 520)]


@pytest.mark.parametrize("m,n,dim", SIZES)
@pytest.mark.parametrize("a", ["codes", "f32", "bf16", "f16"])
def test_product(m, n, dim, a):
    g = gen(m * 7 + n * 3 + dim)
    x = randn(g, m, dim) * torch.exp(randn(g, m, 1))
    y = randn(g, n, dim) * torch.exp(randn(g, n, 1))
    B = sc.byte_quantize(y)
    b_val = R.values(*R.quantize(f64(y)), dim)
    if a != "codes":
        x = x.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[a])
    a_val = R.values(*R.quantize(f64(x)), dim)
    A = sc.byte_quantize(x) if a == "codes" else x
    bias = randn(g, n)
    check_product(A, B, a_val, b_val, dim, bias, torch.float32)
    check_product(A, B, a_val, b_val, dim, None, torch.bfloat16)
    check_product(A, B, a_val, b_val, dim, bias, torch.float16)


@pytest.mark.parametrize("m,n,dim", [(1, 100, 300), (16, 48, 512), (40, 70, 129), (130, 260, 1000), (520, 300, 2048)])
def test_product_of_whole_numbers_is_exact(m, n, dim):
    """Whole numbers up to 14 with a scale of 1/32 (largest 14 = 448 / 32) or 1/64:
    every partial sum is a multiple of 1/4 below 2^20, so any order of additions
    gives the exact sum."""
    g = gen(m + n + dim)

    def rows(k):
        v = torch.randint(0, 15, (k, dim), generator=g, device=DEV).float()
        v[:, ::128] = 14.0
        v *= torch.where(torch.rand(k, dim, generator=g, device=DEV) < 0.5, -1.0, 1.0)
        return v * torch.where(torch.rand(k, 1, generator=g, device=DEV) < 0.5, 0.5, 1.0)

    x, y = rows(m), rows(n)
    want = f64(x) @ f64(y).T
    assert np.abs(want).max() < 2 ** 20
    B = sc.byte_quantize(y)
    assert np.array_equal(f64(sc.byte_dequantize(B)), f64(y))
    assert np.array_equal(f64(sc.byte_product(sc.byte_quantize(x), B)), want)
    assert np.array_equal(f64(sc.byte_product(x, B)), want)


# scale bytes of A and B: the smallest with the largest, products below float32's
# normal range, below its smallest value, and near its largest
@pytest.mark.parametrize("sa,sb", [(0, 246), (246, 0), (1, 126), (60, 60), (62, 40), (40, 60), (0, 110), (0, 0), (236, 100),
                                   (120, 220)])
@pytest.mark.parametrize("m,n,dim", [(2, 64, 256), (20, 65, 2304), (50, 64, 384), (70, 64, 256), (300, 130, 2304),
                                     (2048, 2049, 1152)])
def test_product_at_the_ends_of_the_range(m, n, dim, sa, sb):
    """A term is a multiple of 2^-149 or off by less than one such step, as is
    every sum of such terms below 2^-126 (exact there): dim steps in all, on
    top of the dim 2^-23 of the sums above; the operands' own last bits (see the
    top of this file) times the other operand."""
    r = np.random.default_rng(m + dim + 1000 * sa + sb)

    def rows(k, scale):  # whole groups: padding would have to be zero
        codes = r.integers(0, 127, (k, 128 * R.groups(dim)), dtype=np.uint8)
        codes |= r.integers(0, 2, codes.shape, dtype=np.uint8) << 7
        scales = np.zeros((k, R.scale_bytes(dim)), np.uint8)
        g = R.groups(dim)
        # neighbouring blocks a power of two apart, but for the ends
        scales[:, :g] = np.clip(scale + r.integers(-1, 2, (k, g)), 0, 246)
        return sc.ByteRows(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), dim), codes, scales

    A, ac, as_ = rows(m, sa)
    B, bc, bs = rows(n, sb)
    a, b = R.values(ac[-64:], as_[-64:], dim), R.values(bc[-64:], bs[-64:], dim)
    got = f64(sc.byte_product(A, B)[-64:, -64:])
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    assert mag.max() < 2.0 ** 127 and np.isfinite(got).all()
    tol = (dim + 2) * 2.0 ** -23 * mag + dim * 2.0 ** -149
    small = [2.0 ** -134 * (np.abs(v) < 2.0 ** -130) for v in (a, b)]
    tol += small[0] @ np.abs(b).T + np.abs(a) @ small[1].T + small[0] @ small[1].T
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("m,n,dim", [(4100, 4200, 520), (4090, 4095, 128), (8193, 8000, 1030), (300, 60001, 640)])
def test_product_large(m, n, dim, dtype):
    """Results of many tiles: rows of the first, middle and last ones, whole."""
    g = gen(m + n + dim)
    A, B = (sc.byte_quantize(randn(g, k, dim) * torch.exp(randn(g, k, 1))) for k in (m, n))
    bias = randn(g, n)
    b = R.values(B.codes.cpu().numpy(), B.scales.cpu().numpy(), dim)
    got = sc.byte_product(A, B, bias=bias, dtype=dtype)
    for rows in (slice(0, 3), slice(m // 2 - 2, m // 2 + 2), slice(m - 3, m)):
        a = R.values(A.codes[rows].cpu().numpy(), A.scales[rows].cpu().numpy(), dim)
        want, mag = a @ b.T + f64(bias), np.abs(a) @ np.abs(b).T + np.abs(f64(bias))
        tol = (dim + 2) * 2.0 ** -23 * mag + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.001 + torch.finfo(dtype).tiny
        if dtype != torch.float32:
            tol += 2.0 ** -10 * largest_of_eights(a, b)
        assert (np.abs(f64(got[rows]) - want) <= tol).all()
    for cols in (slice(0, 3), slice(n - 3, n)):  # and a few columns
        a = R.values(A.codes.cpu().numpy(), A.scales.cpu().numpy(), dim)
        want, mag = a @ b[cols].T + f64(bias)[cols], np.abs(a) @ np.abs(b[cols]).T + np.abs(f64(bias))[cols]
        tol = (dim + 2) * 2.0 ** -23 * mag + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.001 + torch.finfo(dtype).tiny
        if dtype != torch.float32:
            tol += 2.0 ** -10 * largest_of_eights(a, b[cols])
        assert (np.abs(f64(got[:, cols]) - want) <= tol).all()


def test_product_float_rows_equal_quantized_rows():
    for m in (1, 2, 7, 16, 17, 64, 65, 200):
        g = gen(m)
        x, B = randn(g, m, 700), sc.byte_quantize(randn(g, 333, 700))
        assert torch.equal(sc.byte_product(x, B), sc.byte_product(sc.byte_quantize(x), B))


@pytest.mark.parametrize("m", [3, 40, 150])
def test_product_strides(m):
    """Rows that are a part of larger buffers, a result inside a larger one."""
    g = gen(m)
    big = sc.byte_quantize(randn(g, 400, 260))
    B = big[37:337]
    x = randn(g, m + 4, 300)[2:2 + m, 11:271]
    C = torch.full((m + 2, 320), 7.0, device=DEV)
    sc.byte_product(x, B, out=C[1:1 + m, 5:305])
    want = sc.byte_product(sc.byte_quantize(x.contiguous()), sc.ByteRows(B.codes.clone(), B.scales.clone(), 260))
    assert torch.equal(C[1:1 + m, 5:305], want)
    C[1:1 + m, 5:305] = 7
    assert bool((C == 7).all())
    codes = torch.zeros(500, 512, dtype=torch.uint8, device=DEV)
    scales = torch.full((500, 16), 99, dtype=torch.uint8, device=DEV)
    wide = sc.ByteRows(codes[9:309, 32:416], scales[9:309, 8:12], 260)
    wide.codes.copy_(B.codes)
    wide.scales.copy_(B.scales)
    assert torch.equal(sc.byte_product(x, wide), want)


@pytest.mark.parametrize("m", [2, 50, 140])
def test_product_non_finite_rows(m):
    g = gen(m)
    x, y = randn(g, m, 300), randn(g, 150, 300)
    x[1, 290], y[149, 3] = float("nan"), float("inf")
    for A in (x, sc.byte_quantize(x)):
        c = sc.byte_product(A, sc.byte_quantize(y))
        nan = torch.isnan(c)
        assert bool(nan[1].all()) and bool(nan[:, 149].all())
        nan[1], nan[:, 149] = False, False
        assert not bool(nan.any())


def test_empty():
    B = sc.byte_quantize(randn(gen(0), 5, 64))
    assert sc.byte_product(randn(gen(0), 0, 64), B).shape == (0, 5)
    assert sc.byte_product(randn(gen(0), 3, 64), B[:0]).shape == (3, 0)
    assert len(sc.byte_quantize(torch.empty(0, 64, device=DEV))) == 0
    assert sc.byte_dequantize(B[:0]).shape == (0, 64)
