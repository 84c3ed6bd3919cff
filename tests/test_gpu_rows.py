"""The row operators on the GPU against the float64 references.

Quantisation and its inverse are exact: codes, scales and values have to be
equal.  Draws are whole numbers and have to be equal.  Products: every term is
exact in float32; a sum of D terms in any order, each addition off by at most
2^-23 of its result (whether the matrix unit rounds or truncates), is off by
at most D 2^-23 sum |a b|; the bias adds one rounding and the result type one
of eps / 2."""
import numpy as np
import pytest
import torch

import soft_clustering_amd as sc
from tests import rows_reference as R

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
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 128), (3, 31), (5, 33), (64, 128), (17, 487), (33, 1000), (2, 8192),
                                      (257, 130)])
def test_quantize_and_back(rows, dim, dtype):
    g = gen(rows * 10007 + dim)
    x = (randn(g, rows, dim) * torch.exp(3 * randn(g, rows, 1))).to(dtype)
    q = sc.mx_quantize(x)
    codes, scales = R.quantize(f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    v = R.values(codes, scales, dim)
    for out in TYPES:
        got = sc.mx_dequantize(q, dtype=out)
        want = torch.from_numpy(v).to(out)  # one rounding; exact but for float16
        assert torch.equal(got.cpu(), want)


def test_quantize_every_border():
    """Grid values, midpoints and their neighbours, at scales from the smallest
    to the largest, subnormals and saturation among them."""
    base = np.array([7.9, 0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5, 7, 7.99], np.float32)
    near = np.concatenate([base, np.nextafter(base, np.float32(9)), np.nextafter(base, np.float32(-9)), -base])
    near = near[: len(near) // 31 * 31].reshape(-1, 31)
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -124, -20, 0, 60, 124, 125):
        for r in near:
            with np.errstate(over="ignore", under="ignore"):
                rows.append(np.concatenate(([np.float32(4)], r)).astype(np.float32) * np.float32(2.0) ** np.float32(e)
                            if e >= -126 else
                            np.ldexp(np.concatenate(([4.0], r.astype(np.float64))), e).astype(np.float32))
    x = np.stack(rows)
    x = x[np.isfinite(x).all(1)]
    q = sc.mx_quantize(torch.from_numpy(x).to(DEV))
    codes, scales = R.quantize(x)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    back = sc.mx_dequantize(q).cpu().numpy()
    assert np.array_equal(back, R.values(codes, scales, 32).astype(np.float32))


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_quantize_non_finite_blocks(dtype):
    x = randn(gen(1), 6, 200).to(dtype)
    x[1, 5], x[2, 40], x[3, 199], x[4] = float("nan"), float("inf"), float("-inf"), 0
    q = sc.mx_quantize(x)
    codes, scales = R.quantize(f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    back = f64(sc.mx_dequantize(q, dtype=dtype))
    assert np.isnan(back[1, :32]).all() and np.isfinite(back[1, 32:]).all()
    assert np.isnan(back[2, 32:64]).all() and np.isnan(back[3, 192:]).all()
    assert (back[4] == 0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_quantize_strides_and_outputs(dtype):
    """Rows of a wider matrix at an odd offset; codes and scales into a part of
    larger buffers, whose other bytes stay as they are."""
    x = randn(gen(2), 40, 300).to(dtype)[3:30, 7:7 + 201]
    want = sc.mx_quantize(x.contiguous())
    codes = torch.full((40, 160), 171, dtype=torch.uint8, device=DEV)
    scales = torch.full((40, 12), 205, dtype=torch.uint8, device=DEV)
    out = sc.MXRows(codes[5:32, 16:144], scales[5:32, 4:12], 201)
    sc.mx_quantize(x, out=out)
    assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
    codes[5:32, 16:144], scales[5:32, 4:12] = 171, 205
    assert bool((codes == 171).all()) and bool((scales == 205).all())
    wide = torch.full((27, 210), 3.0, dtype=dtype, device=DEV)
    sc.mx_dequantize(want, dtype=dtype, out=wide[:, 1:202])
    assert torch.equal(wide[:, 1:202], sc.mx_dequantize(want, dtype=dtype))
    assert bool((wide[:, 0] == 3).all()) and bool((wide[:, 202:] == 3).all())


# ---- products

def check_product(A, B, a_val, b_val, dim, bias, dtype):
    got = sc.mx_product(A, B, bias=bias, dtype=dtype)
    assert got.dtype == dtype
    want = a_val @ b_val.T
    mag = np.abs(a_val) @ np.abs(b_val).T
    if bias is not None:
        want, mag = want + f64(bias)[None], mag + np.abs(f64(bias))[None]
    err = np.abs(f64(got) - want)
    eps = torch.finfo(dtype).eps / 2
    tol = (dim + 2) * 2.0 ** -23 * mag + eps * np.abs(want) * 1.001 + torch.finfo(dtype).tiny
    assert np.isfinite(f64(got)).all()
    worst = (err / tol).max() if err.size else 0.0
    assert worst <= 1, f"error {worst:.3g} of the bound"


SIZES = [(1, 16, 128), (1, 1, 1), (1, 1000, 4096), (5, 33, 100), (16, 129, 1000), (17, 50, 1000), (33, 65, 257),
         (64, 200, 768), (65, 31, 128), (128, 128, 128), (129, 257, 640), (300, 500, 1000), (1024, 300, 96),
         (70, 1, 33), (257, 513, 1152)]


@pytest.mark.parametrize("m,n,dim", SIZES)
@pytest.mark.parametrize("a", ["codes", "f32", "bf16", "f16"])
def test_product(m, n, dim, a):
    g = gen(m * 7 + n * 3 + dim)
    x = randn(g, m, dim) * torch.exp(randn(g, m, 1))
    y = randn(g, n, dim) * torch.exp(randn(g, n, 1))
    B = sc.mx_quantize(y)
    b_val = R.values(*R.quantize(f64(y)), dim)
    if a != "codes":
        x = x.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[a])
    a_val = R.values(*R.quantize(f64(x)), dim)
    A = sc.mx_quantize(x) if a == "codes" else x
    bias = randn(g, n)
    check_product(A, B, a_val, b_val, dim, bias, torch.float32)
    check_product(A, B, a_val, b_val, dim, None, torch.bfloat16)
    check_product(A, B, a_val, b_val, dim, bias, torch.float16)


@pytest.mark.parametrize("m,n,dim", [(1, 100, 300), (16, 48, 512), (40, 70, 129), (130, 260, 1000), (520, 300, 2048)])
def test_product_of_whole_numbers_is_exact(m, n, dim):
    """Grid values at scales 1 and 2: every partial sum is a multiple of 1/4
    below 2^20, so any order of additions gives the exact sum."""
    g = gen(m + n + dim)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6.0], device=DEV)

    def rows(k):
        v = grid[torch.randint(0, 8, (k, dim), generator=g, device=DEV)]
        v[:, ::32] = 4.0  # the block's largest is 4 or 6: its scale is 1
        v *= torch.where(torch.rand(k, dim, generator=g, device=DEV) < 0.5, -1.0, 1.0)
        return v * torch.where(torch.rand(k, 1, generator=g, device=DEV) < 0.5, 2.0, 1.0)

    x, y = rows(m), rows(n)
    want = f64(x) @ f64(y).T
    assert np.abs(want).max() < 2 ** 20
    B = sc.mx_quantize(y)
    assert np.array_equal(f64(sc.mx_product(sc.mx_quantize(x), B)), want)
    assert np.array_equal(f64(sc.mx_product(x, B)), want)


# scale bytes of A and B: the smallest with the largest, products below float32's
# normal range, below its smallest value, and near its largest
@pytest.mark.parametrize("sa,sb", [(0, 254), (254, 0), (1, 126), (60, 60), (62, 40), (40, 60), (0, 110), (0, 0), (254, 100),
                                   (120, 240)])
@pytest.mark.parametrize("m,n,dim", [(2, 64, 256), (20, 65, 2304), (50, 64, 384), (70, 64, 256), (300, 130, 2304),
                                     (4096, 4097, 2176)])
def test_product_at_the_ends_of_the_range(m, n, dim, sa, sb):
    """A term is a multiple of 2^-149 or off by less than one such step, as is
    every sum of such terms below 2^-126 (exact there): dim steps in all, on
    top of the dim 2^-23 of the sums above."""
    r = np.random.default_rng(m + dim + 1000 * sa + sb)

    def rows(k, scale):  # whole groups: padding would have to be zero
        codes = r.integers(0, 256, (k, 64 * R.groups(dim)), dtype=np.uint8)
        # neighbouring blocks a power of two apart, but for the ends
        scales = np.clip(scale + r.integers(-1, 2, (k, 4 * R.groups(dim))), 0, 254).astype(np.uint8)
        return sc.MXRows(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), dim), codes, scales

    A, ac, as_ = rows(m, sa)
    B, bc, bs = rows(n, sb)
    a, b = R.values(ac[-64:], as_[-64:], dim), R.values(bc[-64:], bs[-64:], dim)
    got = f64(sc.mx_product(A, B)[-64:, -64:])
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    assert mag.max() < 2.0 ** 127 and np.isfinite(got).all()
    tol = (dim + 2) * 2.0 ** -23 * mag + dim * 2.0 ** -149
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("m", [2, 40, 70])
def test_product_past_the_range(m):
    """Terms above float32's range: infinite, but where both signs meet, as here
    with a true sum of 0, that sum or no finite number (the matrix unit adds the
    terms of one step before it rounds)."""
    def rows(k, code, scale):
        return sc.MXRows(torch.full((k, 64), code, dtype=torch.uint8, device=DEV),
                         torch.full((k, 4), scale, dtype=torch.uint8, device=DEV), 128)

    B = rows(33, 0x77, 200)
    assert bool((sc.mx_product(rows(m, 0x77, 254), B) == float("inf")).all())
    assert bool((sc.mx_product(rows(m, 0xFF, 254), B) == float("-inf")).all())
    both = sc.mx_product(rows(m, 0xF7, 254), B)
    assert bool(((both == 0) | ~torch.isfinite(both)).all())


def test_product_float_rows_equal_quantized_rows():
    for m in (1, 7, 16, 17, 64, 65, 200):
        g = gen(m)
        x, B = randn(g, m, 700), sc.mx_quantize(randn(g, 333, 700))
        assert torch.equal(sc.mx_product(x, B), sc.mx_product(sc.mx_quantize(x), B))


@pytest.mark.parametrize("m", [3, 40, 150])
def test_product_strides(m):
    """Rows that are a part of larger buffers, a result inside a larger one."""
    g = gen(m)
    big = sc.mx_quantize(randn(g, 400, 260))
    B = big[37:337]
    x = randn(g, m + 4, 300)[2:2 + m, 11:271]
    C = torch.full((m + 2, 320), 7.0, device=DEV)
    sc.mx_product(x, B, out=C[1:1 + m, 5:305])
    want = sc.mx_product(sc.mx_quantize(x.contiguous()), sc.MXRows(B.codes.clone(), B.scales.clone(), 260))
    assert torch.equal(C[1:1 + m, 5:305], want)
    C[1:1 + m, 5:305] = 7
    assert bool((C == 7).all())


@pytest.mark.parametrize("m", [2, 50, 140])
def test_product_non_finite_rows(m):
    g = gen(m)
    x, y = randn(g, m, 300), randn(g, 150, 300)
    x[1, 290], y[149, 3] = float("nan"), float("inf")
    for A in (x, sc.mx_quantize(x)):
        c = sc.mx_product(A, sc.mx_quantize(y))
        nan = torch.isnan(c)
        assert bool(nan[1].all()) and bool(nan[:, 149].all())
        nan[1], nan[:, 149] = False, False
        assert not bool(nan.any())


def test_product_empty():
    B = sc.mx_quantize(randn(gen(0), 5, 64))
    assert sc.mx_product(randn(gen(0), 0, 64), B).shape == (0, 5)
    assert sc.mx_product(randn(gen(0), 3, 64), B[:0]).shape == (3, 0)
    assert len(sc.mx_quantize(torch.empty(0, 64, device=DEV))) == 0
    assert sc.mx_dequantize(B[:0]).shape == (0, 64)
    assert sc.draw(torch.empty(0, 9, device=DEV), torch.empty(0, device=DEV)).shape == (0,)


# ---- draws

SETTINGS = [
    {}, {"temperature": 0.3}, {"temperature": 5.0}, {"temperature": 0.0}, {"top_k": 1}, {"top_k": 5}, {"top_k": 300},
    {"top_p": 0.1}, {"top_p": 0.6}, {"top_p": 0.95}, {"top_p": 0.0}, {"min_p": 0.2}, {"min_p": 1.0}, {"min_p": 3.0},
    {"temperature": 0.7, "top_k": 40, "top_p": 0.9, "min_p": 0.01}, {"temperature": 1.5, "top_k": 2000, "top_p": 0.5},
]


def check_draws(z, u, **kw):
    def row(v, n):  # settings are float32 (top_k whole)
        return float(v[n]) if isinstance(v, torch.Tensor) else float(np.float32(v))

    got = sc.draw(z, u, **kw).cpu().numpy()
    zn, un = f64(z), f64(u)
    want = np.array([R.draw(zn[n], un[n], **{k: (int(row(v, n)) if k == "top_k" else row(v, n))
                                              for k, v in kw.items()}) for n in range(len(un))])
    bad = np.flatnonzero(got != want)
    assert bad.size == 0, f"rows {bad[:5]}: {got[bad[:5]]} instead of {want[bad[:5]]}"


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 2), (40, 63), (9, 256), (30, 257), (20, 1000), (20, 1024), (12, 1025),
                                        (12, 4096), (7, 5001), (6, 16384), (5, 16385), (3, 50001), (2, 131071)])
def test_draw(rows, width, dtype):
    g = gen(rows + width)
    z = (3 * randn(g, rows, width)).to(dtype)
    u = torch.rand(rows, generator=g, device=DEV)
    for kw in SETTINGS:
        check_draws(z, u, **kw)


@pytest.mark.parametrize("width", [100, 1000, 3000, 9000, 40000])
def test_draw_settings_of_each_row(width):
    g = gen(width)
    n = 24
    z, u = 2 * randn(g, n, width), torch.rand(n, generator=g, device=DEV)
    r = torch.rand(n, 4, generator=g, device=DEV)
    t = torch.where(r[:, 0] < 0.2, 0.0, 2 * r[:, 0])
    k = torch.where(r[:, 1] < 0.3, -1.0, r[:, 1] * width / 4).to(torch.int32)
    p = torch.where(r[:, 2] < 0.3, 1.0, r[:, 2])
    m = torch.where(r[:, 3] < 0.3, 0.0, r[:, 3] / 4)
    check_draws(z, u, temperature=t.contiguous(), top_k=k, top_p=p.contiguous(), min_p=m.contiguous())
    check_draws(z, u, temperature=0.9, top_k=k, top_p=0.8)


@pytest.mark.parametrize("width", [64, 900, 3000, 12000, 70000])
def test_draw_ties(width):
    """Few distinct values, so every cut falls among ties and is made by index;
    also rows of one value, and zeros of both signs, which are equal."""
    g = gen(width)
    z = torch.randint(-3, 3, (8, width), generator=g, device=DEV).float() / 2
    z[1], z[2] = 4.0, torch.where(torch.rand(width, generator=g, device=DEV) < 0.5, -0.0, 0.0)
    u = torch.rand(8, generator=g, device=DEV)
    for kw in [{}, {"temperature": 0.0}, {"top_k": width // 3 + 1}, {"top_k": 7}, {"top_p": 0.5}, {"top_p": 0.07},
               {"top_k": width // 2, "top_p": 0.5}, {"top_k": 50, "top_p": 0.99, "min_p": 0.5}]:
        check_draws(z, u, **kw)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("width", [50, 1000, 2500, 10000, 40001])
def test_draw_masked_rows(width, dtype):
    """-inf and the type's lowest value in masked places, rows that the mask
    leaves one value or nothing, NaN and +inf."""
    g = gen(width)
    z = (2 * randn(g, 12, width)).to(dtype)
    low = torch.finfo(dtype).min
    mask = torch.rand(12, width, generator=g, device=DEV) < 0.7
    z[:4] = torch.where(mask[:4], torch.tensor(float("-inf"), dtype=dtype, device=DEV), z[:4])
    z[4:6] = torch.where(mask[4:6], torch.tensor(low, dtype=dtype, device=DEV), z[4:6])
    z[6], z[7] = float("-inf"), low
    z[8], z[8, width - 3] = float("-inf"), -5.0
    z[9, width // 2], z[10, width - 1], z[11, 0] = float("nan"), float("inf"), float("-inf")
    u = torch.rand(12, generator=g, device=DEV)
    for kw in SETTINGS:
        check_draws(z, u, **kw)
    assert sc.draw(z, u)[[6, 9, 10]].tolist() == [-1, -1, -1]


@pytest.mark.parametrize("width", [10, 700, 5000, 33000])
def test_draw_random_numbers_at_the_ends(width):
    z = randn(gen(width), 6, width)
    z[:, -1] = float("-inf")
    u = torch.tensor([0.0, -1.0, 1.0, 2.0, float("nan"), 1 - 2.0 ** -24], device=DEV)
    check_draws(z, u)
    check_draws(z, u, top_k=3)
    check_draws(z, u, top_p=0.5, temperature=0.5)


@pytest.mark.parametrize("width", [500, 20000])
def test_draw_extreme_logits_and_temperatures(width):
    g = gen(width)
    z = randn(g, 10, width)
    z[0] *= 1e37
    z[1] *= 1e-40
    z[2] += 1e6
    z[3] = -3e38 + 1e32 * z[3]
    u = torch.rand(10, generator=g, device=DEV)
    for t in (1.0, 1e-30, 1e30, float("inf"), 1e-3):
        for kw in ({}, {"top_k": 20}, {"top_p": 0.3}, {"top_k": 100, "top_p": 0.9, "min_p": 0.05}):
            check_draws(z, u, temperature=t, **kw)


def test_draw_frequencies():
    """Draws of one row follow its weights: with n draws each count is within
    6 standard deviations of n p."""
    z = torch.tensor([[0.0, 1.0, -1.0, 2.0, 0.5]], device=DEV).expand(200_000, 5).contiguous()
    u = torch.rand(200_000, generator=gen(3), device=DEV)
    ids = sc.draw(z, u, temperature=0.8)
    n = torch.bincount(ids.long(), minlength=5).double().cpu().numpy()
    w = R.kept(f64(z[0]), temperature=0.8)
    p = w / w.sum()
    assert (np.abs(n - 200_000 * p) < 6 * np.sqrt(200_000 * p * (1 - p))).all()


def test_draw_strides():
    g = gen(4)
    big = randn(g, 30, 3000)
    z = big[3:20, 5:2006]
    u = torch.rand(17, generator=g, device=DEV)
    check_draws(z, u, top_k=30, top_p=0.9)
    assert torch.equal(sc.draw(z, u, top_p=0.9), sc.draw(z.contiguous(), u, top_p=0.9))


# ---- together, and how they are called

def test_head_and_draw_together():
    """A run as in serving: rows against stored components, then a component
    for each row from the logits."""
    g = gen(5)
    B = sc.mx_quantize(randn(g, 5000, 384) / 384 ** 0.5)
    bias = randn(g, 5000)
    for m in (1, 20, 100):
        x, u = randn(g, m, 384), torch.rand(m, generator=g, device=DEV)
        logits = sc.mx_product(x, B, bias=bias)
        a = R.values(*R.quantize(f64(x)), 384)
        b = R.values(B.codes.cpu().numpy(), B.scales.cpu().numpy(), 384)
        tol = 386 * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T + np.abs(f64(bias)))
        assert (np.abs(f64(logits) - (a @ b.T + f64(bias))) <= tol).all()
        check_draws(logits, u, temperature=0.8, top_k=50, top_p=0.9, min_p=0.02)


def test_graph_capture_and_replay():
    """The run captured once and replayed on new inputs, with eager work and
    synchronizations between the replays."""
    g = gen(6)
    B = sc.mx_quantize(randn(g, 3000, 256) / 16)
    x, u = randn(g, 80, 256), torch.rand(80, generator=g, device=DEV)

    def work():
        logits = sc.mx_product(x, B)
        return logits, sc.draw(logits, u, top_k=40, top_p=0.9)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, ids = work()
    for i in range(5):
        x.copy_(randn(g, 80, 256))
        u.copy_(torch.rand(80, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want_l, want_i = work()
        assert torch.equal(logits, want_l) and torch.equal(ids, want_i)


def test_streams():
    """Calls on two streams at once, each on its own inputs."""
    g = gen(7)
    B = sc.mx_quantize(randn(g, 4000, 512) / 22)
    xs = [randn(g, 100, 512) for _ in range(2)]
    us = [torch.rand(100, generator=g, device=DEV) for _ in range(2)]
    want = []
    for x, u in zip(xs, us):
        l = sc.mx_product(x, B)
        want.append((l, sc.draw(l, u, top_p=0.8)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                l = sc.mx_product(xs[i], B)
                got[i] = (l, sc.draw(l, us[i], top_p=0.8))
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_the_same_twice():
    g = gen(8)
    x, B = randn(g, 300, 1000), sc.mx_quantize(randn(g, 2000, 1000))
    a, b = sc.mx_product(x, B), sc.mx_product(x, B)
    assert torch.equal(a, b)
    z, u = randn(g, 50, 30000), torch.rand(50, generator=g, device=DEV)
    assert torch.equal(sc.draw(z, u, top_p=0.9), sc.draw(z, u, top_p=0.9))


def test_binding_refusals():
    x = randn(gen(9), 4, 128)
    B = sc.mx_quantize(x)
    with pytest.raises(ValueError, match="rows of"):
        sc.mx_product(randn(gen(9), 4, 100), B)
    with pytest.raises(ValueError, match="contiguous"):
        sc.mx_quantize(x.t())
    with pytest.raises(ValueError, match="overlap"):
        sc.mx_quantize(x[:1].expand(4, 128))
    with pytest.raises(ValueError, match="bias"):
        sc.mx_product(x, B, bias=x[0])
    with pytest.raises(TypeError, match="bias"):
        sc.mx_product(x, B, bias=x[0, :4].double())
    with pytest.raises(TypeError, match="dtype"):
        sc.mx_product(x, B, dtype=torch.float64)
    with pytest.raises(ValueError, match="shape"):
        sc.mx_product(x, B, out=torch.empty(4, 5, device=DEV))
    u = torch.rand(4, device=DEV)
    with pytest.raises(TypeError, match="u must"):
        sc.draw(x, u.double())
    with pytest.raises(ValueError, match="u must"):
        sc.draw(x, u[:3])
    with pytest.raises(TypeError, match="top_k"):
        sc.draw(x, u, top_k=u)
    with pytest.raises(ValueError, match="top_p"):
        sc.draw(x, u, top_p=u[:2])
    with pytest.raises(sc.GMMError, match="temperature"):
        sc.draw(x, u, temperature=-1.0)
    with pytest.raises(TypeError, match="out"):
        sc.draw(x, u, out=torch.empty(4, dtype=torch.int64, device=DEV))


def test_gradients_are_refused_or_off():
    x = randn(gen(10), 4, 128)
    B, bias, u = sc.mx_quantize(x), randn(gen(11), 4), torch.rand(4, device=DEV)
    want, ids = sc.mx_product(x, B, bias=bias), sc.draw(x, u)
    x.requires_grad_(), bias.requires_grad_()
    with pytest.raises(ValueError, match="A requires"):
        sc.mx_product(x, B)
    with pytest.raises(ValueError, match="X requires"):
        sc.mx_quantize(x)
    assert torch.equal(sc.draw(x, u), ids)
    assert torch.equal(sc.mx_product(x.detach(), B, bias=bias.detach()), want)
    with torch.no_grad():
        assert torch.equal(sc.mx_product(x, B, bias=bias), want)
        assert torch.equal(sc.mx_quantize(x).codes, B.codes)


def test_results_over_inputs_are_refused():
    g = gen(12)
    x, u = randn(g, 6, 128), torch.rand(6, generator=g, device=DEV)
    B = sc.mx_quantize(randn(g, 128, 128))
    k, t = torch.full((6,), 3, dtype=torch.int32, device=DEV), torch.ones(6, device=DEV)
    kept = x.clone()
    for call in (lambda: sc.mx_product(x, B, out=x), lambda: sc.mx_product(x[:4], B, out=x[2:]),
                 lambda: sc.mx_product(x, B, bias=x[5], out=x.new_empty(0).set_(x.untyped_storage(), 0, (6, 128), (128, 1))),
                 lambda: sc.draw(x, u, top_k=k, out=k), lambda: sc.draw(x, u, out=u.view(torch.int32)),
                 lambda: sc.draw(x, u, temperature=t, out=t.view(torch.int32)),
                 lambda: sc.draw(x, u, out=x[1, 3:9].view(torch.int32)),
                 lambda: sc.mx_dequantize(B[:8], out=B.codes.view(-1)[:8 * 128 * 4].view(torch.float32).view(8, 128)),
                 lambda: sc.mx_quantize(x, out=sc.MXRows(x.view(torch.uint8)[:, :64], B.scales[:6], 128))):
        with pytest.raises(ValueError, match="shares memory"):
            call()
    assert torch.equal(x, kept)
    # neighbours in one buffer do not overlap
    both = torch.zeros(6, 256, device=DEV)
    both[:, :128] = x
    assert torch.equal(sc.mx_product(both[:, :128], B, out=both[:, 128:]), sc.mx_product(x, B))
