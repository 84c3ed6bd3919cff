"""The losses over rows of logits where their kernels change: lists of every
length, rows divided over workgroups, rows past the caches and past 32 bits,
calls from captured graphs and other streams, and the row operators together."""
import pytest
import torch

import soft_clustering_amd as sc
from tests import losses_reference as R
from tests.test_gpu_losses import (DEV, NAMES, TYPES, check_balance, check_distill, close, gen, lists, randn, rounding,
                                   taken)

pytestmark = pytest.mark.gpu


# by 16 lanes (also with 32 elements each: 8192 rows of 16-bit logits), a wave, 4
# and 16 waves, held and not, divided
@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,V,k", [(8200, 257, 3), (8192, 512, 64), (8193, 511, 9), (8193, 1023, 64), (9000, 1024, 1), (8192, 300, 65), (1030, 4097, 9),
                                   (1024, 16383, 2), (1025, 8200, 200), (300, 16390, 5), (300, 65537, 20),
                                   (280, 131080, 12), (260, 200001, 4), (256, 65536, 1), (255, 65543, 3)])
def test_distill_forms(n, V, k, dtype):
    g = gen(n + V)
    z = (torch.randn(n, V, generator=g, device=DEV, dtype=torch.float32) * 3).to(dtype)
    ids = torch.randint(0, V, (n, k), generator=g, device=DEV)
    ids[torch.rand(n, k, generator=g, device=DEV) < 0.1] = -1
    ids[::7, 0], ids[1::7, k - 1] = V - 1, 0
    teacher = randn(g, n, k).to(dtype)
    some = torch.randperm(n, generator=g, device=DEV)[:40].sort().values  # these against the reference
    some[0], some[-1] = 0, n - 1
    w = torch.rand(n, generator=g, device=DEV) + 0.1
    losses, grad = sc.distill_grad(z, ids, teacher, w, temperature=1.25)
    ref = R.distill(z[some], ids[some], teacher[some], 1.25, w[some])
    close(losses[some], ref[0], ref[1], "losses")
    close(grad[some], ref[2], ref[3] + rounding(dtype, ref[2]), "gradient")
    leaf = z.detach().requires_grad_()
    out = sc.distill(leaf, ids, teacher, 1.25)
    auto, = torch.autograd.grad(out, leaf, w)
    close(out.detach()[some], ref[0], ref[1], "losses for autograd")
    close(auto[some], ref[2], ref[3] + rounding(dtype, ref[2]), "gradient by autograd")
    # every row: the two ways differ by their bounds at most (each is within one)
    far = R.distill(z[:64], ids[:64], teacher[:64], 1.25, w[:64])
    assert bool(((auto[:64].double() - grad[:64].double()).abs() <= 2 * (far[3] + rounding(dtype, far[2]))).all())
    assert torch.equal(sc.distill_grad(z, ids, teacher, w, temperature=1.25)[1], grad)  # the same again


@pytest.mark.parametrize("dtype,V", [(torch.float32, 57345), (torch.float32, 57346), (torch.float32, 57348),
                                     (torch.bfloat16, 114689), (torch.float16, 114695), (torch.bfloat16, 114696),
                                     (torch.float32, 524288 + 3), (torch.bfloat16, 2 ** 20), (torch.float32, 2 ** 20 - 1)])
def test_distill_divided_rows_with_little_left(dtype, V):
    """A last part of a few elements; listed places on both sides of every border."""
    g = gen(V)
    z = (randn(g, 3, V) * 2).to(dtype)
    step = 1024 if dtype == torch.float32 else 2048
    edges = torch.arange(step, V, step, device=DEV)
    at = torch.cat((edges - 1, edges, torch.tensor([V - 1, V - 2, V - 5, V - 8, V - 9], device=DEV))).unique()
    at = at[torch.randperm(len(at), generator=g, device=DEV)][:1024]
    at[:5] = torch.tensor([V - 1, V - 2, V - 5, V - 8, V - 9], device=DEV)
    ids = at[None].repeat(3, 1)
    w = torch.ones(3, device=DEV)
    check_distill(z, ids, randn(g, 3, len(at)).to(dtype), 1.0, w)


@pytest.mark.parametrize("n,V,k", [(4, 300, 64), (3, 900, 400), (2, 16000, 1024), (300, 70000, 1024), (2, 70000, 1024),
                                   (3, 2 ** 20, 1024)])
def test_distill_ids_that_share_bits(n, V, k):
    """Ids a power of two apart, some of them listed several times."""
    g = gen(n + V)
    z = randn(g, n, V)
    far, near = (torch.randint(0, m, (n, k), generator=g, device=DEV) for m in (40, 60))
    ids = (far * 32768 + near) % V
    ids[:, k // 2] = -1
    check_distill(z, ids, randn(g, n, k), 1.0, torch.ones(n, device=DEV))


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,K,k", [(32, 256, 2), (31, 257, 200), (128, 1024, 64), (129, 1024, 1), (500, 1029, 2), (3000, 4102, 1), (8192, 16, 1),
                                   (8193, 16, 1), (1, 1024, 1024), (131, 7, 3), (40000, 7, 2), (5, 16384, 1),
                                   (300, 40001, 2), (2, 2 ** 20, 5), (3, 2 ** 20 - 3, 1000)])
def test_balance_forms(n, K, k, dtype):
    """A small batch in one workgroup, and just above its limits."""
    g = gen(n + 3 * K + k)
    z = (randn(g, n, K) * 2 + randn(g, 1, K)).to(dtype)
    ids, weight = taken(g, z, min(k, K), wide=n % 2 == 0), 64.0 if dtype == torch.float16 else 0.5
    check_balance(z, ids, weight)
    assert all(torch.equal(a, b) for a, b in zip(sc.balance_grad(z, ids, weight), sc.balance_grad(z, ids, weight)))


def test_gradients_past_the_caches_equal_their_parts():
    """256 MB of gradients and more leave in another way."""
    g = gen(7)
    for dtype, n, V in ((torch.float32, 70_000, 1000), (torch.bfloat16, 8200, 16384), (torch.float16, 1100, 131_071)):
        z = torch.randn(n, V, generator=g, device=DEV, dtype=dtype)
        ids = torch.randint(0, V, (n, 5), generator=g, device=DEV)
        teacher = randn(g, n, 5).to(dtype)
        losses, grad = sc.distill_grad(z, ids, teacher, 0.5)
        part = (n + 1) // 2
        for s in (0, n - part):
            one = sc.distill_grad(z[s:s + part], ids[s:s + part], teacher[s:s + part], 0.5)
            assert torch.equal(losses[s:s + part], one[0]) and torch.equal(grad[s:s + part], one[1])
        some = torch.tensor([0, 1, n // 2, n - 1], device=DEV)
        ref = R.balance(z, ids[:, :2], 1.0) if V * n < 10 ** 8 else None
        loss, counts, grad = sc.balance_grad(z, ids[:, :2])
        assert torch.equal(counts, torch.bincount(ids[:, :2].flatten(), minlength=V))
        if ref:
            assert abs(float(loss) - float(ref[0])) <= float(ref[1])
            close(grad[some], ref[3][some], ref[4][some] + rounding(dtype, ref[3][some]), "gradient")
        del ref


def test_rows_past_32_bits():
    """More than 2^33 elements, more workgroups than one dimension of a grid is
    given: the rows at both ends as by themselves."""
    n, V = (1 << 21) + 7, 4100
    g = gen(9)
    z = torch.zeros(n, V, dtype=torch.bfloat16, device=DEV)
    ends = torch.cat((torch.arange(40, device=DEV), torch.arange(n - 40, n, device=DEV)))
    z[ends] = torch.randn(80, V, generator=g, device=DEV).bfloat16()
    ids = torch.randint(0, V, (n, 2), generator=g, device=DEV, dtype=torch.int32)
    teacher = torch.randn(n, 2, generator=g, device=DEV)
    losses = sc.distill(z, ids, teacher)
    some = torch.cat((ends, ends.new_tensor([n // 2, n // 3])))
    ref = R.distill(z[some], ids[some], teacher[some])
    close(losses[some], ref[0], ref[1], "losses")
    losses, grad = sc.distill_grad(z, ids, teacher)
    close(losses[some], ref[0], ref[1], "losses in one pass")
    close(grad[some], ref[2], ref[3] + rounding(z.dtype, ref[2]), "gradient")
    del grad
    leaf = z.requires_grad_()
    auto, = torch.autograd.grad(sc.distill(leaf, ids, teacher).sum(), leaf)
    close(auto[some], ref[2], ref[3] + rounding(z.dtype, ref[2]), "gradient by autograd")
    del auto
    z.requires_grad_(False)
    loss, counts, grad = sc.balance_grad(z, ids, 2.0 ** 30)
    assert torch.equal(counts, torch.bincount(ids.flatten().long(), minlength=V))
    # 80 rows have logits, the others are even over the components: d = the mean count
    c = counts.double()
    p = torch.softmax(z[some].double(), 1)
    d = (p * c).sum(1, keepdim=True)
    scale = V / (2.0 * n * n)
    want = 2.0 ** 30 * scale * p * (c - d)
    # d is off by at most depth(V) + 36 half steps of itself, c - d by one more; an eighth of p, 3.5 * 3 ln 2 * 12 half steps
    bound = 2.0 ** 30 * scale * p * ((c - d).abs() * 200 + d * (R.depth(V) + 200)) * R.U
    close(grad[some], want, bound + rounding(z.dtype, want), "gradient of the balance")
    total = d[:80].sum() + (n - 80) * c.mean()
    assert abs(float(loss) - float(scale * total)) <= float(loss) * (R.depth(V) + 200) * R.U


# ---- refusals, streams and graphs

def test_gradients_that_are_not_computed_are_refused():
    z = torch.randn(4, 50, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    teacher = torch.randn(4, 2, device=DEV)
    leaf = z.clone().requires_grad_()
    for logits in (z, leaf):
        with pytest.raises(ValueError, match="teacher requires"):
            sc.distill(logits, ids, teacher.clone().requires_grad_())
    with pytest.raises(ValueError, match="weights requires"):
        sc.distill_grad(z, ids, teacher, torch.ones(4, device=DEV, requires_grad=True))
    warm = torch.tensor(2.0, requires_grad=True)
    for call in (lambda: sc.distill(z, ids, teacher, warm), lambda: sc.distill(leaf, ids, teacher, warm),
                 lambda: sc.distill_grad(z, ids, teacher, temperature=warm)):
        with pytest.raises(ValueError, match="temperature requires"):
            call()
    with pytest.raises(ValueError, match="weight requires"):
        sc.balance_grad(z, ids, warm)
    first, = torch.autograd.grad(sc.distill(leaf, ids, teacher).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        first.sum().backward()
    out = sc.distill(leaf, ids, teacher).sum() + sc.balance(leaf, ids)[0]
    with torch.no_grad():
        leaf.add_(1)  # the backward would read other logits than the forward did
    with pytest.raises(RuntimeError, match="modified"):
        out.backward()


def test_two_streams_at_once():
    g = gen(11)
    sets = []
    for n, V in ((3, 60000), (2, 90001)):  # divided rows: with a workspace
        z = randn(g, n, V)
        ids, teacher = lists(g, z, 30)
        sets.append((z, ids, teacher))
    want = [(sc.distill_grad(*s), sc.balance_grad(s[0], s[1])) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, a in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append((sc.distill_grad(*a), sc.balance_grad(a[0], a[1])))
    torch.cuda.synchronize()
    for i, (d, b) in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(d, want[i % 2][0]))
        assert all(torch.equal(x, y) for x, y in zip(b, want[i % 2][1]))


@pytest.mark.parametrize("n,V", [(20, 100), (300, 1000), (3, 50000), (700, 20000)])
def test_captured_and_replayed(n, V):
    """Two graphs of the losses and their gradients, replayed in turn on new logits
    with eager work between."""
    g = gen(n + V)
    z = randn(g, n, V)
    ids, teacher = lists(g, z, 8)

    def work():
        leaf = z.detach().requires_grad_()
        losses = sc.distill(leaf, ids, teacher, 2.0)
        loss, counts = sc.balance(leaf, ids)
        grad, = torch.autograd.grad(losses.mean() + 0.1 * loss, leaf)
        return (losses.detach(), loss.detach(), counts, grad) + sc.distill_grad(z, ids, teacher, 1 / n, 2.0) \
            + sc.balance_grad(z, ids, 0.1)

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
        z.copy_(randn(g, n, V))
        ids.copy_(torch.randint(-1, V, ids.shape, generator=g, device=DEV))
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        kept = [r.clone() for pair in results for r in pair]
        want = work()
        torch.cuda.synchronize()
        for i, r in enumerate(kept):
            assert torch.equal(r, want[i % len(want)]), (turn, i)


# ---- together

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=NAMES.get)
@pytest.mark.parametrize("n,K,D", [(300, 700, 96), (130, 16500, 200)])
def test_the_row_operators_together(n, K, D, dtype):
    """Means held in 8 bits score a batch of points (the mixture's logits, the
    teacher's); a model's logits are trained on the best of them and on balance;
    points are drawn for it; the means after a step are held in 8 bits again.
    Everything against float64 from the same stored values."""
    g = gen(n + K + D)
    x, means = randn(g, n, D), randn(g, K, D)
    held = sc.byte_quantize(means)
    values = sc.byte_dequantize(held).double()
    bias = (values ** 2).sum(1).div(-2).float()
    scores = sc.byte_product(x, held, bias=bias)
    xq = sc.byte_dequantize(sc.byte_quantize(x)).double()
    want = xq @ values.t().contiguous() + bias.double()
    mag = xq.abs() @ values.abs().t().contiguous() + bias.abs().double()
    assert bool(((scores.double() - want).abs() <= (D + 3) * 2.0 ** -23 * mag).all())
    teacher, ids = torch.topk(scores, 20, dim=1)
    W = (randn(g, D, K) / D).requires_grad_()
    logits = (x @ W).to(dtype)
    picked = sc.draw(logits.detach(), torch.rand(n, generator=g, device=DEV))
    assert int(picked.min()) >= 0
    losses = sc.distill(logits, ids, teacher, 2.0)
    even, counts = sc.balance(logits, picked)
    total = losses.mean() + 0.01 * even
    step, = torch.autograd.grad(total, W)
    z = logits.detach()
    d, b = R.distill(z, ids, teacher, 2.0, torch.full((n,), 1 / n, device=DEV)), R.balance(z, picked, 0.01)
    close(losses.detach(), d[0], d[1], "losses")
    assert abs(float(even) - float(b[0])) <= float(b[1]) and torch.equal(counts, b[2])
    # two gradients, each rounded to the type of the logits, and their rounded sum
    each = d[3] + b[4] + rounding(dtype, d[2]) + rounding(dtype, b[3])
    each = each + rounding(dtype, d[2].abs() + b[3].abs() + each)
    left = x.double().t().contiguous()
    got = left @ (d[2] + b[3])
    # the product over n points in float32 (the gradient is widened before it), n 2^-23 of the magnitudes
    bound = left.abs() @ each + (n + 2) * 2.0 ** -23 * (left.abs() @ ((d[2] + b[3]).abs() + each))
    close(step, got, bound, "gradient of the weights")
    after = sc.byte_quantize((means + 0.1 * randn(g, K, D)), out=held)
    assert after is held and not torch.equal(sc.byte_dequantize(held).double(), values)


@pytest.mark.parametrize("V", [3, 40000, 2 ** 20])
def test_no_rows_of_any_width(V):
    z, ids = torch.empty(0, V, device=DEV), torch.empty(0, 3, dtype=torch.int64, device=DEV)
    losses, grad = sc.distill_grad(z, ids, torch.empty(0, 3, device=DEV))
    assert losses.shape == (0,) and grad.shape == (0, V)
    assert sc.distill(z, ids, torch.empty(0, 3, device=DEV)).shape == (0,)
    loss, counts, grad = sc.balance_grad(z, ids)
    assert float(loss) == 0 and counts.shape == (V,) and not bool(counts.any()) and grad.shape == (0, V)
