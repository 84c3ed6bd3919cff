"""Distillation and balance on the GPU against the float64 references; the bounds
are derived in losses_reference.py, and a gradient is rounded once to the type of
the logits (half a step, at least of the smallest number)."""
import math

import pytest
import torch

import soft_clustering_amd as sc
from tests import losses_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}
INF, NAN = float("inf"), float("nan")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def rounding(t, want):
    info = torch.finfo(t)
    return info.eps / 2 * want.abs() * 1.001 + info.tiny * info.eps


def close(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        at = tuple(i)
        raise AssertionError(f"{what}: {int(bad.sum())} off, first at {i}: {float(got[at])} for {float(want[at])}, "
                             f"bound {float(bound[at])}")


def lists(g, z, k, wide=True):
    """A teacher's top k of noisy logits, some shorter."""
    n, V = z.shape
    both = z.float() + randn(g, n, V)
    top = torch.topk(both, k, dim=1)
    ids = top.indices
    short = torch.randint(0, k + 1, (n, 1), generator=g, device=DEV)
    cut = (torch.rand(n, 1, generator=g, device=DEV) < 0.3) & (torch.arange(k, device=DEV)[None, :] >= short)
    ids = torch.where(cut, -1, ids)
    return ids if wide else ids.int(), top.values.to(z.dtype)


def check_distill(z, ids, teacher, T, weights):
    losses, bound, grad, bounds = R.distill(z, ids, teacher, T, weights)
    got, got_grad = sc.distill_grad(z, ids, teacher, weights, temperature=T)
    assert got.dtype == torch.float32 and got_grad.dtype == z.dtype
    close(got, losses, bound, "losses in one pass")
    close(got_grad, grad, bounds + rounding(z.dtype, grad), "gradient in one pass")
    leaf = z.detach().requires_grad_()
    out = sc.distill(leaf, ids, teacher, T)
    close(out.detach(), losses, bound, "losses")
    auto, = torch.autograd.grad(out, leaf, weights)
    close(auto, grad, bounds + rounding(z.dtype, grad), "gradient")
    with torch.no_grad():
        close(sc.distill(leaf, ids, teacher, T), losses, bound, "losses without a gradient")


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 3, 1), (5, 31, 7), (64, 64, 64), (7, 65, 33), (130, 100, 8), (9, 1000, 64),
          (300, 1023, 5), (257, 1024, 16), (33, 1025, 65), (20, 2049, 100), (6, 4100, 300), (11, 5000, 1), (3, 9000, 1024),
          (2, 16384, 40), (5, 16385, 64), (3, 20001, 1000), (1, 131071, 64), (70, 131072, 8), (300, 33000, 16), (2, 262147, 9)]


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,V,k", SHAPES)
def test_distill(n, V, k, dtype):
    g = gen(n + 7 * V + k)
    z = (randn(g, n, V) * 4).to(dtype)
    ids, teacher = lists(g, z, k, wide=(n + V) % 2 == 0)
    check_distill(z, ids, teacher, 1.0, torch.rand(n, generator=g, device=DEV) + 0.1)


@pytest.mark.parametrize("T", [0.05, 0.7, 2.0, 30.0])
@pytest.mark.parametrize("n,V,k", [(40, 700, 20), (4, 20000, 50)])
def test_distill_temperatures(n, V, k, T):
    g = gen(V + k)
    z = randn(g, n, V) * 5 + 100
    ids, teacher = lists(g, z, k)
    check_distill(z, ids, teacher, T, randn(g, n))


@pytest.mark.parametrize("n,V,k", [(50, 300, 12), (8, 3000, 200), (4, 40000, 1024)])
def test_distill_ids_listed_twice(n, V, k):
    g = gen(V)
    z = randn(g, n, V) * 3
    ids = torch.randint(0, V, (n, k), generator=g, device=DEV)
    ids[:, 1::2] = ids[:, 0::2]
    ids[0] = 5
    ids[1, : k // 2] = -1
    check_distill(z, ids, randn(g, n, k), 1.5, torch.ones(n, device=DEV))


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("V", [200, 1500, 20000])
def test_distill_masked_logits(V, dtype):
    """Components that the model (or the teacher) has masked: -inf, or the lowest
    number of the type."""
    g = gen(V)
    n, k = 12, 10
    z = (randn(g, n, V) * 3).to(dtype)
    low = torch.finfo(dtype).min
    ids, teacher = lists(g, z, k)
    teacher[0, 3:] = -INF
    teacher[1, 1] = low
    teacher[2] = low              # even over the list
    teacher[11] = -INF            # nothing listed
    keep = torch.zeros(n, V, dtype=torch.bool, device=DEV).scatter_(1, ids.clamp(min=0), True)
    for row, masked in ((3, -INF), (4, low)):
        z[row] = torch.where(keep[row], z[row], torch.tensor(masked, dtype=dtype, device=DEV))
    z[5] = low                    # even over the row
    z[6, : V // 2] = torch.where(keep[6, : V // 2], z[6, : V // 2], torch.tensor(low, dtype=dtype, device=DEV))
    z[11] = NAN                   # whatever its logits
    ref = z.clone()
    ref[11] = 0
    losses, bound, grad, bounds = R.distill(ref, ids, teacher, 1.0)
    got, got_grad = sc.distill_grad(z, ids, teacher)
    close(got, losses, bound, "losses")
    close(got_grad, grad, bounds + rounding(dtype, grad), "gradient")
    assert float(got[11]) == 0 and not bool(got_grad[11].any())
    leaf = z.detach().requires_grad_()
    out = sc.distill(leaf, ids, teacher)
    auto, = torch.autograd.grad(out.sum(), leaf)
    close(auto, grad, bounds + rounding(dtype, grad), "gradient by autograd")
    assert float(out[11]) == 0


@pytest.mark.parametrize("V", [100, 3000, 20000])
def test_distill_rows_without_an_answer(V):
    """They are NaN throughout, and the rows between them are as without them."""
    g = gen(V)
    n, k = 16, 6
    z = randn(g, n, V)
    ids, teacher = lists(g, z, k)
    ids[:, 0] = torch.arange(n, device=DEV)
    want = sc.distill_grad(z, ids, teacher)
    bad = [1, 3, 5, 7, 9, 11]
    z[1, V - 1], z[3, 0], z[5] = NAN, INF, -INF
    teacher[7, 0], teacher[9, 0] = NAN, INF
    ids[11, 0] = V
    for big in (V, 2 ** 31 - 1, 2 ** 40):
        ids[11, 0] = big
        got, grad = sc.distill_grad(z, ids, teacher)
        leaf = z.detach().requires_grad_()
        out = sc.distill(leaf, ids, teacher)
        auto, = torch.autograd.grad(out.sum(), leaf)
        for a, b in ((got, grad), (out.detach(), auto)):
            assert bool(torch.isnan(a[bad]).all()) and bool(torch.isnan(b[bad]).all())
            ok = [i for i in range(n) if i not in bad]
            assert torch.equal(a[ok], want[0][ok])
            assert bool(torch.isfinite(b[ok]).all())


def test_distill_listed_component_without_weight():
    """A listed component whose own logit is -inf: an infinite loss, a gradient all
    the same; no share in the teacher: nothing lost."""
    z = torch.zeros(2, 10, device=DEV)
    z[:, 4] = -INF
    ids = torch.tensor([[4, 1], [4, 1]], device=DEV)
    teacher = torch.tensor([[0.0, 0.0], [-300.0, 0.0]], device=DEV)
    losses, grad = sc.distill_grad(z, ids, teacher)
    assert float(losses[0]) == INF and abs(float(losses[1]) - math.log(9)) < 1e-6
    want = torch.full((2, 10), 1 / 9, dtype=torch.float64, device=DEV)
    want[:, 4] = 0
    want[0, 4], want[0, 1] = -0.5, 1 / 9 - 0.5
    want[1, 1] = 1 / 9 - 1
    assert float((grad - want).abs().max()) < 1e-6


def test_distill_differences():
    """The gradient against differences of the float64 loss."""
    g = gen(3)
    z = randn(g, 4, 30)
    ids, teacher = lists(g, z, 5)
    w = torch.rand(4, generator=g, device=DEV)
    grad = sc.distill_grad(z, ids, teacher, w, temperature=1.7)[1].double()
    h = 1e-5
    for v in range(30):
        step = torch.zeros(4, 30, dtype=torch.float64, device=DEV)
        step[:, v] = h
        up, down = (R.distill(z.double() + s * step, ids, teacher, 1.7)[0] for s in (1, -1))
        assert float(((up - down) / (2 * h) * w - grad[:, v]).abs().max()) < 1e-6


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_distill_strides(dtype):
    """Rows of wider matrices at odd offsets, a gradient inside a larger one,
    weights broadcast by autograd."""
    g = gen(9)
    big = (randn(g, 40, 900) * 3).to(dtype)
    z = big[3:33, 7:7 + 701]
    ids, teacher = lists(g, z.contiguous(), 9)
    wide_ids = torch.full((30, 20), -7, device=DEV)
    wide_ids[:, 5:14] = ids
    wide_teacher = torch.zeros(30, 31, dtype=dtype, device=DEV)
    wide_teacher[:, 11:20] = teacher
    want, want_grad = sc.distill_grad(z.contiguous(), ids, teacher, 0.25, temperature=1.3)
    room = torch.full((32, 720), 3.0, dtype=dtype, device=DEV)
    got, grad = sc.distill_grad(z, wide_ids[:, 5:14], wide_teacher[:, 11:20], 0.25, temperature=1.3,
                                out=room[1:31, 5:706])
    assert torch.equal(got, want) and torch.equal(grad, want_grad)
    room[1:31, 5:706] = 3
    assert bool((room == 3).all())
    leaf = big.detach().requires_grad_()
    sc.distill(leaf[3:33, 7:708], ids, teacher, 1.3).mean().backward()  # one weight for all rows, by expansion
    part = leaf.grad[3:33, 7:708].double() * 30 * 0.25
    ref = R.distill(z, ids, teacher, 1.3, torch.full((30,), 0.25, device=DEV))
    close(part, ref[2], ref[3] * 1.5 + 2 * rounding(dtype, ref[2]) + 8 * torch.finfo(dtype).tiny * torch.finfo(dtype).eps,
          "gradient of a mean")
    assert not bool(leaf.grad[0].any()) and not bool(leaf.grad[:, :7].any())


# ---- balance

def taken(g, z, k, wide):
    ids = torch.topk(z.float() + randn(g, *z.shape), k, dim=1).indices
    ids[torch.rand(len(ids), generator=g, device=DEV) < 0.2] = -1
    if k > 1:
        ids[::5, 1] = -1
    return ids if wide else ids.int()


def check_balance(z, ids, weight):
    loss, bound, counts, grad, bounds = R.balance(z, ids, weight)
    got, got_counts, got_grad = sc.balance_grad(z, ids, weight)
    assert got.dtype == torch.float32 and got.shape == () and got_grad.dtype == z.dtype
    assert got_counts.dtype == torch.int64 and torch.equal(got_counts, counts)
    assert abs(float(got) - float(loss)) <= float(bound)
    close(got_grad, grad, bounds + rounding(z.dtype, grad), "gradient in one pass")
    leaf = z.detach().requires_grad_()
    out, out_counts = sc.balance(leaf, ids)
    assert torch.equal(out_counts, counts) and not out_counts.requires_grad
    assert abs(float(out) - float(loss)) <= float(bound)
    auto, = torch.autograd.grad(weight * out, leaf)
    close(auto, grad, bounds + rounding(z.dtype, grad), "gradient")
    with torch.no_grad():
        assert abs(float(sc.balance(leaf, ids)[0]) - float(loss)) <= float(bound)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,K,k", [(1, 1, 1), (2, 2, 2), (5, 3, 2), (64, 8, 2), (33, 31, 7), (1000, 64, 2), (300, 65, 1),
                                   (257, 1000, 3), (4100, 1024, 1), (700, 1025, 16), (129, 2049, 4), (50, 4100, 8),
                                   (20, 5001, 64), (65, 16384, 4), (30, 16385, 5), (9, 65536, 3), (7, 70001, 1000),
                                   (20000, 16, 1), (66000, 5, 3)])
def test_balance(n, K, k, dtype):
    g = gen(n + 3 * K + k)
    z = (randn(g, n, K) * 2 + randn(g, 1, K)).to(dtype)
    check_balance(z, taken(g, z, min(k, K), wide=(n + K) % 2 == 0), 100.0 if dtype == torch.float16 else 0.5)


def test_balance_of_drawn_ids():
    """One id for a row, as draw gives them: -1 for a row without a distribution,
    which counts for nothing."""
    g = gen(5)
    z = randn(g, 500, 300)
    z[7], z[9, 3] = -INF, NAN
    ids = sc.draw(z, torch.rand(500, generator=g, device=DEV))
    assert int(ids[7]) == int(ids[9]) == -1
    loss, counts, grad = sc.balance_grad(z, ids)
    ref = z.clone()
    ref[[7, 9]] = 0
    want = R.balance(ref, ids)
    assert abs(float(loss) - float(want[0])) <= float(want[1]) and torch.equal(counts, want[2])
    close(grad, want[3], want[4] + rounding(z.dtype, want[3]), "gradient")
    assert not bool(grad[[7, 9]].any())
    spread = torch.full((500, 6), 99, dtype=torch.int32, device=DEV)
    spread[:, 2] = ids
    again = sc.balance_grad(z, spread[:, 2])
    assert torch.equal(again[1], counts) and torch.equal(again[2], grad) and torch.equal(again[0], loss)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("K", [64, 1500, 20000])
def test_balance_masked_logits(K, dtype):
    g = gen(K)
    z = (randn(g, 40, K) * 2).to(dtype)
    ids = taken(g, z, 3, True)
    keep = torch.zeros(40, K, dtype=torch.bool, device=DEV).scatter_(1, ids.clamp(min=0), True)
    low = torch.finfo(dtype).min
    for row, masked in ((1, -INF), (2, low), (3, -INF)):
        z[row, : K // 2] = torch.where(keep[row, : K // 2], z[row, : K // 2], torch.tensor(masked, dtype=dtype, device=DEV))
    z[4] = low
    check_balance(z, ids, 64.0)


@pytest.mark.parametrize("K", [64, 1500, 20000])
def test_balance_without_an_answer(K):
    g = gen(K)
    z = randn(g, 30, K)
    ids = taken(g, z, 2, True)
    none = torch.full_like(ids, -1)
    loss, counts, grad = sc.balance_grad(z, none)
    assert float(loss) == 0 and not bool(counts.any()) and not bool(grad.any())
    want = sc.balance(z, ids)[1]
    for bad in (K, 2 ** 31 - 1, 2 ** 40):
        worse = torch.cat((ids, torch.full((30, 1), -1, device=DEV)), 1)
        worse[8, 2] = bad
        loss, counts, grad = sc.balance_grad(z, worse)
        assert math.isnan(float(loss)) and bool(torch.isnan(grad[8]).all()) and torch.equal(counts, want)
    ids[6, 0] = 1
    z[6] = -INF
    loss, _, grad = sc.balance_grad(z, ids)
    assert math.isnan(float(loss)) and bool(torch.isnan(grad[6]).all())
    assert bool(torch.isfinite(grad[[i for i in range(30) if i != 6]]).all())


def test_balance_differences():
    g = gen(4)
    z = randn(g, 6, 20)
    ids = taken(g, z, 2, False)
    grad = sc.balance_grad(z, ids, 3.0)[2].double()
    h = 1e-5
    for n in range(6):
        for e in range(20):
            step = torch.zeros(6, 20, dtype=torch.float64, device=DEV)
            step[n, e] = h
            up, down = (float(R.balance(z.double() + s * step, ids)[0]) for s in (1, -1))
            assert abs(3 * (up - down) / (2 * h) - float(grad[n, e])) < 1e-6


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_balance_strides(dtype):
    g = gen(9)
    big = (randn(g, 60, 900) * 3).to(dtype)
    z = big[3:43, 7:7 + 701]
    ids = taken(g, z, 3, False)
    wide = torch.full((40, 9), 5, dtype=torch.int32, device=DEV)
    wide[:, 4:7] = ids
    want = sc.balance_grad(z.contiguous(), ids, 50.0)
    room = torch.full((42, 720), 3.0, dtype=dtype, device=DEV)
    got = sc.balance_grad(z, wide[:, 4:7], 50.0, out=room[1:41, 5:706])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    room[1:41, 5:706] = 3
    assert bool((room == 3).all())


def test_empty():
    z = torch.empty(0, 9, device=DEV)
    ids = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    losses, grad = sc.distill_grad(z, ids, torch.empty(0, 2, device=DEV))
    assert losses.shape == (0,) and grad.shape == (0, 9)
    leaf = z.detach().requires_grad_()
    sc.distill(leaf, ids, torch.empty(0, 2, device=DEV)).sum().backward()
    assert leaf.grad.shape == (0, 9)
    loss, counts, grad = sc.balance_grad(z, ids)
    assert float(loss) == 0 and counts.tolist() == [0] * 9 and grad.shape == (0, 9)
    leaf = z.detach().requires_grad_()
    sc.balance(leaf, ids)[0].backward()
    assert leaf.grad.shape == (0, 9)
