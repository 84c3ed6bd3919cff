"""The row operators where their kernels change: every tile of the products,
draws of rows that are split, sorted or searched by ranges, results past the
caches, offsets past 32 bits, and calls that share memory or streams.

Everything here is exact: whole-number products, draws, and the same call made
in two ways."""
import numpy as np
import pytest
import torch

import soft_clustering_amd as sc
from soft_clustering_amd import ivf_probe
from tests import rows_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def whole(g, n, dim):
    """Grid values at scale 1 or 2: 4-bit rows hold them exactly, and every
    partial sum of products is a multiple of 1/4."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6.0], device=DEV)
    v = grid[torch.randint(0, 8, (n, dim), generator=g, device=DEV)]
    v[:, ::32] = 4.0
    v *= torch.where(torch.rand(n, dim, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    return v * torch.where(torch.rand(n, 1, generator=g, device=DEV) < 0.5, 2.0, 1.0)


# ---- products

# rows of A that fill few tiles, tiles of 256 x 128 and of 256 x 256; groups
# below 4, odd and even, a last group of one value; results past the caches
@pytest.mark.parametrize("m,n,dim", [(65, 129, 513), (300, 38405, 100), (300, 38405, 385), (257, 33000, 700),
                                     (1000, 33001, 1153), (4096, 4096, 2049), (4001, 4300, 2500), (3841, 3969, 4096),
                                     (8192, 8320, 200), (8192, 8320, 1000), (8192, 8320, 2100), (8191, 8321, 130)])
def test_every_tile(m, n, dim):
    g = gen(m + n + dim)
    x, y = whole(g, m, dim), whole(g, n, dim)
    want = x.double() @ y.double().t().contiguous()
    assert float(want.abs().max()) < 2 ** 20
    B, bias = sc.mx_quantize(y), torch.randint(-50, 50, (n,), generator=g, device=DEV).float()
    assert torch.equal(sc.mx_product(x, B).double(), want)
    got = sc.mx_product(sc.mx_quantize(x), B, bias=bias, dtype=torch.bfloat16)
    assert torch.equal(got, (want + bias.double()).float().bfloat16())


@pytest.mark.parametrize("m", [70, 600])
@pytest.mark.parametrize("groups", [4, 5, 7])
def test_product_of_strided_codes(m, groups):
    """Codes and scales whose rows lie in wider buffers, scales at every
    multiple of 4 bytes."""
    g = gen(m + groups)
    dim = 128 * groups - 3
    x, y = whole(g, m, dim), whole(g, 40000, dim)
    A, B = sc.mx_quantize(x), sc.mx_quantize(y)

    def inside(q, pad):
        codes = torch.full((len(q), 64 * groups + 16 * pad), 255, dtype=torch.uint8, device=DEV)
        scales = torch.full((len(q), 4 * groups + 4 * pad), 255, dtype=torch.uint8, device=DEV)
        out = sc.MXRows(codes[:, 16 * (pad - 1):16 * (pad - 1) + 64 * groups],
                        scales[:, 4 * (pad - 1):4 * (pad - 1) + 4 * groups], dim)
        out.codes.copy_(q.codes)
        out.scales.copy_(q.scales)
        return out

    want = (x.double() @ y.double().t().contiguous())
    for pad in (1, 2, 3):
        assert torch.equal(sc.mx_product(inside(A, pad), inside(B, 4 - pad)).double(), want)


def test_strides_past_the_limit_are_refused():
    far = 2 ** 23 + 16
    codes = torch.zeros(far + 64, dtype=torch.uint8, device=DEV).as_strided((2, 64), (far, 1))
    scales = torch.zeros(2, 4, dtype=torch.uint8, device=DEV)
    rows = sc.MXRows(codes, scales, 100)
    with pytest.raises(sc.GMMError, match="code stride"):
        sc.mx_product(torch.zeros(2, 100, device=DEV), rows)
    with pytest.raises(sc.GMMError, match="code stride"):
        sc.mx_dequantize(rows)


# ---- large rows and offsets

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,dim", [(70001, 300), (9001, 5119), (3, 2 ** 20), (33, 2 ** 20 - 5)])
def test_large_dequantisation_equals_its_parts(rows, dim, dtype):
    x = randn(gen(rows), rows, dim, dtype=torch.bfloat16)
    q = sc.mx_quantize(x)
    codes, scales = R.quantize(f64(x[-3:]))
    assert np.array_equal(q.codes[-3:].cpu().numpy(), codes) and np.array_equal(q.scales[-3:].cpu().numpy(), scales)
    wide = torch.full((rows, dim + 3), 5.0, dtype=dtype, device=DEV)
    sc.mx_dequantize(q, dtype=dtype, out=wide[:, 1:dim + 1])
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, dim + 1:] == 5).all())
    part = max(1, (1 << 20) // dim)
    for s in range(0, rows, part):
        assert torch.equal(wide[s:s + part, 1:dim + 1], sc.mx_dequantize(q[s:s + part], dtype=dtype))


def test_quantize_past_32_bits():
    """More elements than one launch takes, offsets past 2^33."""
    rows, dim = 1_048_700, 8192
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device=DEV)
    g = gen(1)
    some = [0, 262_140, 524_280, 1_048_560, rows - 128]  # 1_048_576 rows are one launch
    for s in some:
        x[s:s + 128] = randn(g, 128, dim, dtype=torch.bfloat16)
    q = sc.mx_quantize(x)
    for s in some:
        part = sc.mx_quantize(x[s:s + 128])
        assert torch.equal(q.codes[s:s + 128], part.codes) and torch.equal(q.scales[s:s + 128], part.scales)
    x.fill_(9)
    sc.mx_dequantize(q, dtype=torch.bfloat16, out=x)
    for s in some:
        assert torch.equal(x[s:s + 128], sc.mx_dequantize(q[s:s + 128], dtype=torch.bfloat16))
    assert not bool(x[1000:100_000].any()) and not bool(x[600_000:700_000].any())


def test_product_past_32_bits():
    g = gen(2)
    x, y = whole(g, 70_000, 64), whole(g, 65_003, 64)
    A, B = sc.mx_quantize(x), sc.mx_quantize(y)
    c = sc.mx_product(A, B)
    for rows in (slice(0, 300), slice(66_000, 66_100), slice(69_900, 70_000)):
        assert torch.equal(c[rows], sc.mx_product(A[rows], B))
    assert torch.equal(c[:, 64_990:].double(), x.double() @ y[64_990:].double().t().contiguous())


def test_few_rows_past_32_bits():
    """Stored codes of over 2^32 bytes, read by the few-rows kernel."""
    n, g = 68_000_000, gen(3)
    codes = torch.randint(0, 256, (n, 64), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(126, 129, (n, 4), generator=g, device=DEV, dtype=torch.uint8)
    B = sc.MXRows(codes, scales, 128)
    x = whole(g, 2, 128)
    c = sc.mx_product(x, B)
    for s in (0, 33_000_000, n - 5000):
        y = sc.mx_dequantize(B[s:s + 5000])
        assert torch.equal(c[:, s:s + 5000].double(), x.double() @ y.double().t().contiguous())


# ---- draws

def reference(z, u, **kw):
    z, u = f64(z), f64(u)
    kw = {k: (v if k == "top_k" else float(np.float32(v))) for k, v in kw.items()}
    return [R.draw(z[n], u[n], **kw) for n in range(len(u))]


CUTS = [{}, {"temperature": 0.0}, {"min_p": 0.1}, {"top_k": 1}, {"top_k": 50}, {"top_k": 700, "top_p": 0.9},
        {"top_k": 1500}, {"top_k": 2048, "top_p": 0.8, "min_p": 0.001}, {"top_k": 2049}, {"top_k": 3001, "top_p": 0.7},
        {"top_k": 15000}, {"top_p": 0.05}, {"top_p": 0.5, "temperature": 3.0}, {"top_p": 0.999}]


@pytest.mark.parametrize("width", [16385, 20000, 70001])
@pytest.mark.parametrize("kind", ["normal", "flat", "ties", "steep"])
def test_draw_of_few_long_rows(width, kind):
    """Rows split over workgroups; flat rows put thousands of elements in one
    bin of the cut, ties more than any list holds."""
    g = gen(width)
    z = randn(g, 6, width)
    if kind == "flat":
        z *= 1e-4
    elif kind == "ties":
        z = torch.round(z)
    elif kind == "steep":
        z *= 30
    z[4, ::3] = float("-inf")
    z[5] = float("-inf")
    u = torch.rand(6, generator=g, device=DEV)
    for kw in CUTS:
        assert sc.draw(z, u, **kw).tolist() == reference(z, u, **kw), kw


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 33, 64, 127, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_split_rows_equal_whole_rows(rows, dtype):
    """The same rows among many are not split."""
    g = gen(rows)
    z = (2 * randn(g, 150, 30011)).to(dtype)
    z[0, 5] = float("nan")
    u = torch.rand(150, generator=g, device=DEV)
    for kw in CUTS:
        assert torch.equal(sc.draw(z[:rows], u[:rows], **kw), sc.draw(z, u, **kw)[:rows]), kw


@pytest.mark.parametrize("width", [20001, 131072])
def test_draw_of_long_rows_with_settings_of_each(width):
    g = gen(width)
    n = 40
    z, u = 2 * randn(g, n, width), torch.rand(n, generator=g, device=DEV)
    r = torch.rand(n, 4, generator=g, device=DEV)
    t = torch.where(r[:, 0] < 0.2, 0.0, 2 * r[:, 0])
    k = torch.where(r[:, 1] < 0.3, 0.0, r[:, 1] ** 4 * width).to(torch.int32)
    p = torch.where(r[:, 2] < 0.3, 1.0, r[:, 2])
    m = torch.where(r[:, 3] < 0.3, 0.0, r[:, 3] / 8)
    got = sc.draw(z, u, temperature=t, top_k=k, top_p=p, min_p=m)
    want = [R.draw(f64(z[i]), float(u[i]), float(t[i]), int(k[i]), float(p[i]), float(m[i])) for i in range(n)]
    assert got.tolist() == want


@pytest.mark.parametrize("width", [100, 256, 700, 1024])
@pytest.mark.parametrize("rows", [4096, 12_289, 40_003])
def test_draw_of_many_short_rows(rows, width):
    """Settings of each row, some with cuts and some without: they are drawn
    by different kernels, several rows to a wave."""
    g = gen(rows + width)
    z, u = 2 * randn(g, rows, width), torch.rand(rows, generator=g, device=DEV)
    z[5], z[77, 3], z[78, 0] = float("-inf"), float("nan"), float("inf")
    r = torch.rand(rows, 4, generator=g, device=DEV)
    t = torch.where(r[:, 0] < 0.1, 0.0, 2 * r[:, 0])
    k = torch.where(r[:, 1] < 0.7, 0.0, r[:, 1] * width / 3).to(torch.int32)
    p = torch.where(r[:, 2] < 0.7, 1.0, r[:, 2])
    m = torch.where(r[:, 3] < 0.5, 0.0, r[:, 3] / 8)
    got = sc.draw(z, u, temperature=t, top_k=k, top_p=p, min_p=m)
    for s in range(0, rows, 4000):  # fewer rows: one kernel, a wave to each
        e = slice(s, min(s + 4000, rows))
        one = sc.draw(z[e], u[e], temperature=t[e].clone(), top_k=k[e].clone(), top_p=p[e].clone(), min_p=m[e].clone())
        assert torch.equal(got[e], one)
    zs, us = f64(z[:120]), f64(u[:120])
    want = [R.draw(zs[i], us[i], float(t[i]), int(k[i]), float(p[i]), float(m[i])) for i in range(120)]
    assert got[:120].tolist() == want
    plain = sc.draw(z, u)
    assert plain[:120].tolist() == [R.draw(zs[i], us[i]) for i in range(120)]
    assert torch.equal(plain[-90:], sc.draw(z[-90:], u[-90:]))


@pytest.mark.parametrize("width", [60, 1000, 3000, 12_000, 20_000])
def test_smallest_temperatures(width):
    """Down to the smallest float32: only the largest logits have weight."""
    g = gen(width)
    z = torch.round(4 * randn(g, 4, width)) / 4
    z[1] *= 1e-38
    z[2] = 0
    u = torch.rand(4, generator=g, device=DEV)
    for t in (1e-35, 1e-37, 1e-38, 1e-42, 1.5e-45):
        for kw in ({}, {"top_k": 1}, {"top_k": 3}, {"top_p": 0.4}):
            assert sc.draw(z, u, temperature=t, **kw).tolist() == reference(z, u, temperature=t, **kw), (t, kw)


def test_draw_past_32_bits():
    g = gen(4)
    z = torch.zeros(4200, 2 ** 20, dtype=torch.bfloat16, device=DEV)
    for s in (0, 2100, 4190):
        z[s:s + 10] = 2 * randn(g, 10, 2 ** 20, dtype=torch.bfloat16)
    u = torch.rand(4200, generator=g, device=DEV)
    for kw in ({}, {"top_k": 40, "top_p": 0.9}, {"top_p": 0.6}):
        ids = sc.draw(z, u, **kw)
        for s in (0, 2100, 4190):
            assert torch.equal(ids[s:s + 10], sc.draw(z[s:s + 10], u[s:s + 10], **kw))
    z = z.view(-1)[:4_300_000 * 1000].view(4_300_000, 1000)
    z[-100:] = 2 * randn(g, 100, 1000, dtype=torch.bfloat16)
    u = torch.rand(4_300_000, generator=g, device=DEV)
    for kw in ({}, {"top_k": 5}):
        ids = sc.draw(z, u, **kw)
        assert torch.equal(ids[-100:], sc.draw(z[-100:], u[-100:], **kw))


def test_draw_of_very_many_rows():
    """More rows than 4 to a wave of the largest launch."""
    n = (1 << 27) + 77
    z = torch.zeros(n, 2, dtype=torch.bfloat16, device=DEV)
    z[::3, 1], z[1::3, 0] = float("-inf"), float("-inf")
    u = torch.zeros(n, device=DEV)
    u[2::3] = 0.75
    for kw in ({}, {"top_p": 0.99}):
        ids = sc.draw(z, u, **kw)
        assert not bool(ids[::3].any()) and bool((ids[1::3] == 1).all()) and bool((ids[2::3] == 1).all())


def test_equal_weights_divide_evenly():
    """V equal logits and u = (i + 1/2) / V draw component i, for every i."""
    for v in (1, 3, 64, 1000, 1024, 4096, 16384, 65536):
        u = ((torch.arange(v, device=DEV, dtype=torch.float64) + 0.5) / v).float()
        pick = torch.unique(torch.linspace(0, v - 1, min(v, 300), device=DEV).long())
        z = torch.full((1, v), 2.5, device=DEV).expand(len(pick), v).contiguous()
        assert torch.equal(sc.draw(z, u[pick]).long(), pick)


def test_rows_past_the_largest_width_are_refused():
    """Among them one whose width is 5 in its low 32 bits."""
    z, u = torch.zeros(1, 2 ** 32 + 5, dtype=torch.bfloat16, device=DEV), torch.full((1,), 0.5, device=DEV)
    for call in (lambda: sc.draw(z, u), lambda: sc.mx_quantize(z)):
        with pytest.raises(ValueError, match="rows of"):
            call()
    with pytest.raises(sc.GMMError, match="V must be"):
        sc.draw(z[:, :2 ** 20 + 1], u)


@pytest.mark.parametrize("width", [1, 1000, 16384, 16385, 131072, 2 ** 20])
def test_draw_of_no_rows(width):
    """Also at the widths whose rows would be split."""
    z, u = torch.empty(0, width, device=DEV), torch.empty(0, device=DEV)
    assert sc.draw(z, u, top_k=3, top_p=0.9).shape == (0,)


# ---- workspaces, graphs and streams

def test_workspace_contents_do_not_matter():
    g = gen(5)
    z, u = randn(g, 5, 60_000), torch.rand(5, generator=g, device=DEV)
    x, B = randn(g, 40, 900), sc.mx_quantize(randn(g, 500, 900))
    want = [sc.draw(z, u, top_p=0.9), sc.draw(z, u, top_k=30), sc.draw(z, u, temperature=0.0), sc.mx_product(x, B)]
    for fill in (0, 255, 127):
        got = []
        for call in (lambda: sc.draw(z, u, top_p=0.9), lambda: sc.draw(z, u, top_k=30),
                     lambda: sc.draw(z, u, temperature=0.0), lambda: sc.mx_product(x, B)):
            # what the call's workspace is then taken from
            blocks = [torch.full((s,), fill, dtype=torch.uint8, device=DEV) for s in (2 ** 15, 2 ** 18, 2 ** 20, 2 ** 22)]
            del blocks
            got.append(call())
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs_and_eager_work_between():
    g = gen(6)
    B = sc.mx_quantize(randn(g, 20_000, 300) / 17)
    x, u = randn(g, 24, 300), torch.rand(24, generator=g, device=DEV)

    def first():
        return sc.draw(sc.mx_product(x, B), u, top_k=40, top_p=0.9)

    def second():
        q = sc.mx_quantize(x)
        return sc.draw(sc.mx_product(q, B, dtype=torch.bfloat16), u, top_p=0.7), sc.mx_dequantize(q)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first(), second()
    torch.cuda.current_stream().wait_stream(side)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        a = first()
    with torch.cuda.graph(two, pool=one.pool()):
        b, back = second()
    for i in range(4):
        x.copy_(randn(g, 24, 300))
        u.copy_(torch.rand(24, generator=g, device=DEV))
        for graph in ((one, two), (two, one))[i % 2]:
            graph.replay()
            if i > 1:
                torch.cuda.synchronize()
        got = [t.clone() for t in (b, back)] if i % 2 == 0 else [a.clone()]
        want = list(second()) if i % 2 == 0 else [first()]
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


def test_split_draws_on_two_streams():
    g = gen(7)
    zs = [randn(g, 3, 100_000) for _ in range(2)]
    us = [torch.rand(3, generator=g, device=DEV) for _ in range(2)]
    want = [sc.draw(z, u, top_p=0.8) for z, u in zip(zs, us)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sc.draw(zs[i], us[i], top_p=0.8))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])


# ---- the compressed scan

def test_compressed_topk():
    g = gen(8)
    n, dim, k = 6000, 128, 10
    X = torch.randint(0, 200, (n, dim), generator=g, device=DEV).float()
    Q = torch.randint(0, 200, (50, dim), generator=g, device=DEV).float()
    rows = sc.mx_quantize(X)
    ids, d = ivf_probe.exact_topk(Q, X, k)
    # the shortlist is everything: the exact result
    all_i, all_d = ivf_probe.compressed_topk(Q, rows, X, k, shortlist=n, batch=16)
    assert torch.equal(all_i, ids) and torch.equal(all_d, d)
    short = 300
    got_i, got_d = ivf_probe.compressed_topk(Q, rows, X, k, shortlist=short)
    x, q, i = f64(X), f64(Q), got_i.cpu().numpy()
    true = ((x[i] - q[:, None]) ** 2).sum(2)
    assert np.array_equal(true, got_d.cpu().numpy())
    # a row that is nearer than the last one returned was not in the shortlist:
    # its score is below the shortlist's last, but for the product's error
    xv, qv = R.values(*R.quantize(x), dim), R.values(*R.quantize(q), dim)
    half = (x ** 2).sum(1) / 2
    score = qv @ xv.T - half
    tol = (dim + 2) * 2.0 ** -23 * (np.abs(qv) @ np.abs(xv).T + half)
    last = np.sort(score, 1)[:, -short]
    dist = ((q[:, None] - x[None]) ** 2).sum(2)
    nearer = dist < true[:, -1:]
    np.put_along_axis(nearer, i, False, 1)
    assert (score[nearer] <= (last[:, None] + 2 * tol)[nearer]).all()
    assert ivf_probe.compressed_topk(Q[:0], rows, X, k)[0].shape == (0, k)


def test_compressed_topk_of_tensors_with_gradients():
    """Its results are whole numbers: nothing to refuse."""
    g = gen(10)
    X = torch.randint(0, 50, (300, 40), generator=g, device=DEV).float()
    rows, want = sc.mx_quantize(X), ivf_probe.exact_topk(X[:5], X, 3)
    got = ivf_probe.compressed_topk(X[:5].clone().requires_grad_(), rows, X.clone().requires_grad_(), 3, 300)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_compressed_topk_with_a_kept_bias():
    """The same results; X is then read at the shortlist alone, whose rows are
    still checked."""
    g = gen(11)
    X = torch.randint(0, 200, (20_000, 96), generator=g, device=DEV).float()
    Q = torch.randint(0, 200, (9, 96), generator=g, device=DEV).float()
    rows, bias = sc.mx_quantize(X), ivf_probe.scan_bias(X)
    want = ivf_probe.compressed_topk(Q, rows, X, 10, 100)
    got = ivf_probe.compressed_topk(Q, rows, X, 10, 100, bias=bias)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    far = torch.topk(sc.mx_product(Q, rows, bias=bias), 101, dim=1).indices.unique()
    left_out = torch.ones(20_000, dtype=torch.bool, device=DEV).index_fill(0, far, False)
    Y = torch.where(left_out[:, None], 0.5, X)   # what no shortlist holds
    got = ivf_probe.compressed_topk(Q, rows, Y, 10, 100, bias=bias)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    Y[want[0][3, 2], 5] += 0.25
    with pytest.raises(ValueError, match="integer values"):
        ivf_probe.compressed_topk(Q, rows, Y, 10, 100, bias=bias)


def test_compressed_topk_with_the_norms_of_the_rows():
    """The shortlist is then what lies nearest to the query among the values
    that the 4-bit rows stand for, query rounded as well: all of it exact, as
    the values are multiples of 2 below 2^8 (scales of 2^0 up), their squares'
    sums below 2^24 and half of those multiples of 1/2."""
    g = gen(13)
    centre = torch.randint(40, 200, (300, 1, 64), generator=g, device=DEV).float()
    X = (centre + torch.randint(-12, 13, (300, 20, 64), generator=g, device=DEV)).reshape(-1, 64)
    Q = X[::71] + torch.randint(-3, 4, (85, 64), generator=g, device=DEV)
    rows, (k, short) = sc.mx_quantize(X), (5, 40)
    bias = ivf_probe.scan_bias(rows)
    xh, qh = f64(sc.mx_dequantize(rows)), f64(sc.mx_dequantize(sc.mx_quantize(Q)))
    assert np.array_equal(f64(bias), (xh ** 2).sum(1) / -2)
    assert torch.equal(ivf_probe.scan_bias(rows, part=1000), bias)
    got, d = ivf_probe.compressed_topk(Q, rows, X, k, short, bias=bias)
    dh = ((qh[:, None] - xh[None]) ** 2).sum(2)
    border = np.sort(dh, 1)[:, short - 1:short]
    exact = ((f64(Q)[:, None] - f64(X)[None]) ** 2).sum(2)
    for i in range(len(Q)):
        inside = np.flatnonzero(dh[i] < border[i])          # in every shortlist; ties at the border may be
        may = np.flatnonzero(dh[i] <= border[i])
        best = np.sort(exact[i, inside])[:k]
        assert set(got[i].tolist()) <= set(may.tolist())
        assert np.array_equal(exact[i, got[i].cpu().numpy()], d[i].cpu().numpy())
        assert (f64(d[i])[:len(best)] <= best).all()


def test_compressed_topk_makes_no_copy_of_the_base():
    """2^21 x 128 values are 1 GiB, 2 GiB in float64."""
    X = torch.randint(0, 200, (2 ** 21, 128), generator=gen(12), device=DEV, dtype=torch.int16).float()
    rows = sc.mx_quantize(X)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    ivf_probe.compressed_topk(X[:1].clone(), rows, X)
    assert torch.cuda.max_memory_allocated() - before < 2 ** 29
    torch.cuda.reset_peak_memory_stats()
    ivf_probe.compressed_topk(X[:1].clone(), rows, X, bias=torch.zeros(2 ** 21, device=DEV))
    # no part of X in float64, 2^24 values or 2^27 bytes: the bias and the scores are 2^23
    # bytes each, and topk, whose memory is the library's, holds a few 2^21 values of 12 bytes
    assert torch.cuda.max_memory_allocated() - before < 2 ** 27


def test_calls_from_two_host_threads():
    import threading

    g = gen(9)
    B = sc.mx_quantize(randn(g, 20_000, 256) / 16)
    xs = [randn(g, n, 256) for n in (5, 90)]
    us = [torch.rand(len(x), generator=g, device=DEV) for x in xs]

    def work(i):
        logits = sc.mx_product(xs[i], B)
        return logits, sc.draw(logits, us[i], top_k=100, top_p=0.9)

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[i].append(work(i))
            stream.synchronize()
        except Exception as e:  # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and [len(v) for v in got] == [20, 20]
    for i in range(2):
        for logits, ids in got[i]:
            assert torch.equal(logits, want[i][0]) and torch.equal(ids, want[i][1])
