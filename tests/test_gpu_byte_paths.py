"""The 8-bit rows where their kernels change: every form of the products, strided
codes, results and rows past the caches and past 32 bits, calls from captured
graphs and other streams, and the search over compressed rows.

Products are of whole numbers or compared with the same call made in two ways, so
that everything is exact: values up to 14 (scales 1/32 or 1/64), products that
are multiples of 1/4 up to 196, so that also of 8 neighbouring ones none has bits
below 2^-13 of the largest (196 * 2^-13 < 1/4), and sums below 2^20."""
import numpy as np
import pytest
import torch

import soft_clustering_amd as sc
from soft_clustering_amd import ivf_probe
from tests import byte_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def whole(g, n, dim):
    v = torch.randint(0, 15, (n, dim), generator=g, device=DEV).float()
    v[:, ::128] = 14.0
    v *= torch.where(torch.rand(n, dim, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    return v * torch.where(torch.rand(n, 1, generator=g, device=DEV) < 0.5, 0.5, 1.0)


# one row of fewer than 8 groups, of 8, of a part of 32, of more than 32; few rows
# with and without quantisation inside, of 16, 32 and 64 to a workgroup, of one
# and two blocks of B rows; tiles of 128 and of 256
@pytest.mark.parametrize("m,n,dim", [(1, 700, 897), (1, 701, 1024), (1, 702, 1500), (1, 703, 4096), (1, 705, 4097),
                                     (1, 9001, 8001), (2, 130, 4001), (5, 9003, 2000), (16, 8193, 512), (17, 300, 1300),
                                     (32, 8200, 130), (33, 8193, 1200), (64, 20001, 300), (65, 129, 513),
                                     (100, 40001, 300), (128, 66003, 140), (129, 33000, 700), (300, 38405, 385),
                                     (1000, 33001, 1153), (4096, 4096, 2049), (3841, 3969, 4001), (4001, 4300, 650)])
def test_every_form(m, n, dim):
    g = gen(m + n + dim)
    x, y = whole(g, m, dim), whole(g, n, dim)
    want = x.double() @ y.double().t().contiguous()
    assert float(want.abs().max()) < 2 ** 20
    A, B, bias = sc.byte_quantize(x), sc.byte_quantize(y), torch.randint(-50, 50, (n,), generator=g, device=DEV).float()
    for a in (A, x, x.bfloat16(), x.half()):
        assert torch.equal(sc.byte_product(a, B).double(), want)
    for dtype in TYPES[1:]:
        assert torch.equal(sc.byte_product(A, B, bias=bias, dtype=dtype), (want + bias.double()).float().to(dtype))


@pytest.mark.parametrize("dim", [1024, 1025, 3333, 4096, 5000])
def test_one_row_equals_its_place_among_two(dim):
    """Normal values: two ways to the same sums, D 2^-23 of the magnitudes apart
    at most for each; rows in 8 bits or quantised on the way give the same."""
    g = gen(dim)
    x, y = randn(g, 2, dim), randn(g, 3001, dim) * torch.exp(3 * randn(g, 3001, 1))
    x[0, 5] *= 1000
    A, B = sc.byte_quantize(x), sc.byte_quantize(y)
    one, two = sc.byte_product(A[:1], B), sc.byte_product(A, B)[:1]
    mag = sc.byte_dequantize(A[:1]).abs().double() @ sc.byte_dequantize(B).abs().double().t().contiguous()
    assert bool(((one - two).abs().double() <= 2 * (dim + 2) * 2.0 ** -23 * mag).all())
    for dtype in TYPES:
        assert torch.equal(sc.byte_product(x[:1].to(dtype), B), sc.byte_product(sc.byte_quantize(x[:1].to(dtype)), B))


@pytest.mark.parametrize("sa,sb", [(0, 246), (246, 0), (1, 126), (60, 60), (40, 60), (0, 0), (236, 100)])
@pytest.mark.parametrize("dim", [1024, 1500, 5000])
def test_one_row_at_the_ends_of_the_range(dim, sa, sb):
    """As for more rows: a term or sum off by one step of 2^-149 at most besides
    the roundings; A's values are held in bfloat16, whose last bit is 2^-133."""
    r = np.random.default_rng(dim + 1000 * sa + sb)

    def rows(k, scale):
        codes = r.integers(0, 127, (k, 128 * R.groups(dim)), dtype=np.uint8)
        codes[:, dim:] = 0
        scales = np.zeros((k, R.scale_bytes(dim)), np.uint8)
        scales[:, :R.groups(dim)] = scale
        return sc.ByteRows(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), dim), \
            R.values(codes, scales, dim)

    (A, a), (B, b) = rows(1, sa), rows(65, sb)
    got, want, mag = f64(sc.byte_product(A, B)), a @ b.T, np.abs(a) @ np.abs(b).T
    assert mag.max() < 2.0 ** 127 and np.isfinite(got).all()
    small = [2.0 ** -134 * (np.abs(v) < 2.0 ** -130) for v in (a, b)]
    tol = (dim + 2) * 2.0 ** -23 * mag + dim * 2.0 ** -149
    tol += small[0] @ np.abs(b).T + np.abs(a) @ small[1].T + small[0] @ small[1].T
    assert (np.abs(got - want) <= tol).all()


def test_one_row_with_blocks_that_are_nan():
    g = gen(8)
    x, y = randn(g, 1, 2000), randn(g, 90, 2000)
    y[7, 1999], y[80, 3] = float("nan"), float("inf")
    B = sc.byte_quantize(y)
    for A in (x, sc.byte_quantize(x)):
        nan = torch.isnan(sc.byte_product(A, B))[0]
        assert nan.nonzero().flatten().tolist() == [7, 80]
    x[0, 1300] = float("-inf")
    for A in (x, sc.byte_quantize(x)):
        assert bool(torch.isnan(sc.byte_product(A, B)).all())


@pytest.mark.parametrize("m", [1, 9, 70, 600])
@pytest.mark.parametrize("groups", [4, 5, 8, 9])
def test_product_of_strided_codes(m, groups):
    g = gen(m + groups)
    dim = 128 * groups - 3
    x, y = whole(g, m, dim), whole(g, 40000, dim)
    A, B = sc.byte_quantize(x), sc.byte_quantize(y)

    def inside(q, pad):
        codes = torch.full((len(q), 128 * groups + 16 * pad), 255, dtype=torch.uint8, device=DEV)
        wide = R.scale_bytes(dim)
        scales = torch.full((len(q), wide + 4 * pad), 255, dtype=torch.uint8, device=DEV)
        out = sc.ByteRows(codes[:, 16 * (pad - 1):16 * (pad - 1) + 128 * groups], scales[:, 4 * (pad - 1):4 * (pad - 1) + wide], dim)
        out.codes.copy_(q.codes)
        out.scales.copy_(q.scales)
        return out

    want = (x.double() @ y.double().t().contiguous())
    for pad in (1, 2, 3):
        assert torch.equal(sc.byte_product(inside(A, pad), inside(B, 4 - pad)).double(), want)


def test_strides_past_the_limit_are_refused():
    far = 2 ** 23 + 16
    codes = torch.zeros(far + 128, dtype=torch.uint8, device=DEV).as_strided((2, 128), (far, 1))
    rows = sc.ByteRows(codes, torch.zeros(2, 4, dtype=torch.uint8, device=DEV), 100)
    with pytest.raises(sc.GMMError, match="code stride"):
        sc.byte_product(torch.zeros(2, 100, device=DEV), rows)
    with pytest.raises(sc.GMMError, match="code stride"):
        sc.byte_dequantize(rows)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("rows,dim", [(70001, 1000), (9001, 5119), (700_001, 100), (3, 2 ** 20), (33, 2 ** 20 - 5)])
def test_large_calls_equal_their_parts(rows, dim, dtype):
    """Also past the caches (256 MB and more)."""
    x = randn(gen(rows), rows, dim, dtype=torch.bfloat16).to(dtype)
    q = sc.byte_quantize(x)
    codes, scales = R.quantize(f64(x[-3:]))
    assert np.array_equal(q.codes[-3:].cpu().numpy(), codes) and np.array_equal(q.scales[-3:].cpu().numpy(), scales)
    wide = torch.full((rows, dim + 3), 5.0, dtype=dtype, device=DEV)
    sc.byte_dequantize(q, dtype=dtype, out=wide[:, 1:dim + 1])
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, dim + 1:] == 5).all())
    part = max(1, (1 << 20) // dim)
    for s in range(0, rows, part):
        one = sc.byte_quantize(x[s:s + part])
        assert torch.equal(one.codes, q.codes[s:s + part]) and torch.equal(one.scales, q.scales[s:s + part])
        assert torch.equal(wide[s:s + part, 1:dim + 1], sc.byte_dequantize(q[s:s + part], dtype=dtype))


def test_quantize_past_32_bits():
    """More elements than one launch takes, offsets past 2^33."""
    rows, dim = 1_048_700, 8192
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device=DEV)
    g = gen(1)
    some = [0, 262_140, 524_280, 1_048_560, rows - 128]
    for s in some:
        x[s:s + 128] = randn(g, 128, dim, dtype=torch.bfloat16)
    q = sc.byte_quantize(x)
    for s in some:
        part = sc.byte_quantize(x[s:s + 128])
        assert torch.equal(q.codes[s:s + 128], part.codes) and torch.equal(q.scales[s:s + 128], part.scales)
    x.fill_(9)
    sc.byte_dequantize(q, dtype=torch.bfloat16, out=x)
    for s in some:
        assert torch.equal(x[s:s + 128], sc.byte_dequantize(q[s:s + 128], dtype=torch.bfloat16))
    assert not bool(x[1000:100_000].any()) and not bool(x[600_000:700_000].any())


def test_products_past_32_bits():
    """A result of over 2^32 elements; stored codes of over 2^32 bytes, read by the
    kernels of few rows and of one."""
    g = gen(2)
    x, y = whole(g, 70_000, 64), whole(g, 65_003, 64)
    A, B = sc.byte_quantize(x), sc.byte_quantize(y)
    for dtype in (torch.float32, torch.bfloat16):
        c = sc.byte_product(A, B, dtype=dtype)
        for rows in (slice(0, 300), slice(66_000, 66_100), slice(69_900, 70_000)):
            assert torch.equal(c[rows], sc.byte_product(A[rows], B, dtype=dtype))
        want = (x.double() @ y[64_990:].double().t().contiguous()).float().to(dtype)
        assert torch.equal(c[:, 64_990:], want)
        del c
    for n, dim in ((36_000_000, 128), (4_300_000, 1024)):
        codes = torch.randint(0, 96, (n, dim), generator=g, device=DEV, dtype=torch.uint8)  # values up to 30
        scales = torch.full((n, R.scale_bytes(dim)), 127, dtype=torch.uint8, device=DEV)
        B = sc.ByteRows(codes, scales, dim)
        x = torch.zeros(2, dim, device=DEV)
        x[0, 3], x[1, dim - 1] = 2.0, -1.0
        for A in (x, x[1:]):
            c = sc.byte_product(A, B)
            for s in (0, n // 2, n - 5000):
                y = sc.byte_dequantize(B[s:s + 5000])
                assert torch.equal(c[:, s:s + 5000].double(), A.double() @ y.double().t().contiguous())


# ---- streams and graphs

def test_two_streams_at_once():
    """Calls that need a workspace each, on two streams."""
    g = gen(5)
    x, y, B = randn(g, 3000, 700), randn(g, 3000, 700), sc.byte_quantize(randn(g, 2000, 700))
    want = [sc.byte_product(v, B, dtype=torch.bfloat16) for v in (x, y)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, v in zip(streams, (x, y)):
            with torch.cuda.stream(s):
                got.append(sc.byte_product(v, B, dtype=torch.bfloat16))
    torch.cuda.synchronize()
    for i, c in enumerate(got):
        assert torch.equal(c, want[i % 2])


@pytest.mark.parametrize("m", [1, 30, 300])
def test_captured_and_replayed(m):
    """Two graphs whose workspaces are apart, replayed in turn on new values with
    eager work between."""
    g = gen(m)
    x, B = randn(g, m, 1100), sc.byte_quantize(randn(g, 900, 1100))
    Q = sc.byte_quantize(x)
    bias = randn(g, 900)

    def work():
        sc.byte_quantize(x, out=Q)
        return sc.byte_product(Q, B, bias=bias), sc.byte_product(x, B, dtype=torch.bfloat16), sc.byte_dequantize(Q)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(work())
        graphs.append(graph)
    for turn in range(5):
        x.copy_(randn(g, m, 1100))
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        kept = [r.clone() for pair in results for r in pair]
        want = work()
        torch.cuda.synchronize()
        for i, r in enumerate(kept):
            assert torch.equal(r, want[i % 3])


# ---- the search over compressed rows

def test_compressed_topk_of_8_bits():
    g = gen(4)
    X = torch.randint(0, 256, (5000, 37), generator=g, device=DEV).float()
    Q = torch.randint(0, 256, (41, 37), generator=g, device=DEV).float()
    rows = sc.byte_quantize(X)
    k, short = 7, 100
    want_i, want_d = ivf_probe.exact_topk(Q, X, k)
    all_i, all_d = ivf_probe.compressed_topk(Q, rows, X, k, shortlist=5000, batch=16)
    assert torch.equal(all_i, want_i) and torch.equal(all_d, want_d)
    bias = ivf_probe.scan_bias(X)
    assert torch.equal(ivf_probe.scan_bias(rows, part=999),
                       (sc.byte_dequantize(rows).double() ** 2).sum(1).div(-2).float())
    for b in (None, bias, ivf_probe.scan_bias(rows)):
        got_i, got_d = ivf_probe.compressed_topk(Q, rows, X, k, shortlist=short, bias=b)
        # by the same steps: the product, its best, their exact distances
        for i in range(len(Q)):
            scores = sc.byte_product(Q, rows, bias=bias if b is None else b)[i]
            cand = torch.topk(scores, short).indices
            d2 = ((X[cand] - Q[i]).double() ** 2).sum(1).long()
            order = sorted(zip(d2.tolist(), cand.tolist()))[:k]
            assert got_i[i].tolist() == [c for _, c in order] and got_d[i].tolist() == [d for d, _ in order]
    assert ivf_probe.recall(got_i, want_i)[0] > 0.9
    assert ivf_probe.compressed_topk(Q[:0], rows, X, k)[0].shape == (0, k)
