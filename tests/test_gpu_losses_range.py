"""The losses over the whole range of finite logits and of temperatures: masks of
large numbers over stretches that fill a lane's vectors, a wave or a divided part,
rows of nothing else, logits far from 0, and exponents on both sides of the
magnitude at which the kernels form them in another way.  The bounds are those of
losses_reference.py, which hold for any of it: an exponent is off by a part of its
distance from the row's largest, whatever the logits' size."""
import math

import pytest
import torch

import soft_clustering_amd as sc
from tests import losses_reference as R
from tests.test_gpu_losses import DEV, NAMES, TYPES, check_balance, check_distill, close, gen, lists, randn, rounding, taken

pytestmark = pytest.mark.gpu

# shorter than a vector, 16 lanes, a wave, 4 and 16 waves, whole long rows, divided, past what a thread holds
FORMS = [(12, 3), (12, 200), (12, 1000), (12, 1500), (12, 4097), (12, 16384), (12, 16390), (300, 40001), (5, 40001),
         (256, 70000)]
MASKS = {torch.float32: (-1e9, -1e10, -1e12, -1e20, -1e30), torch.bfloat16: (-1e9, -1e12, -1e30),
         torch.float16: (-6e4,)}


def masked(g, n, V, dtype, mask):
    """Rows of which stretches, or all, have a mask; what is left free."""
    at = torch.arange(V, device=DEV)
    shapes = [at < V // 2, at >= V // 2, (at < V // 3) | (at > V // 3 + 10), at % 2 == 0, at >= 0, at < V - 1, at >= 1,
              (at // 8) % 2 == 0, at < 0]
    hidden = torch.stack(shapes)[torch.arange(n, device=DEV) % len(shapes)]
    z = (randn(g, n, V) * 3).to(dtype)
    return torch.where(hidden, torch.tensor(mask, device=DEV).to(dtype), z), hidden


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,V", FORMS)
def test_distill_masks(n, V, dtype):
    g = gen(V)
    for mask in MASKS[dtype]:
        z, hidden = masked(g, n, V, dtype, mask)
        ids, teacher = lists(g, z, min(V, 9))
        free = hidden.any(1, keepdim=True) & ~hidden.gather(1, ids.clamp(min=0))
        ids = torch.where(free | hidden.all(1, keepdim=True), ids, -1)
        check_distill(z, ids, teacher, 1.0, torch.rand(n, generator=g, device=DEV) + 0.1)
        # a masked component is listed
        ids[:, 0] = torch.randint(0, V, (n,), generator=g, device=DEV)
        check_distill(z, ids, randn(g, *ids.shape).to(dtype), 1.0, torch.rand(n, generator=g, device=DEV) + 0.1)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,K", FORMS)
def test_balance_masks(n, K, dtype):
    g = gen(K)
    for mask in MASKS[dtype]:
        z, _ = masked(g, n, K, dtype, mask)
        check_balance(z, taken(g, z, min(K, 3), wide=True), 64.0)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("T", [2.0 ** -60, 1e-12, 1e-9, 1e-6, 2.0 ** 60])
def test_distill_temperatures(T, dtype):
    for n, V in FORMS:
        g = gen(V)
        z = (randn(g, n, V) * 3).to(dtype)
        ids, teacher = lists(g, z, min(V, 9))
        w = torch.rand(n, generator=g, device=DEV) + 0.1
        if dtype != torch.float16 or T < 1:
            check_distill(z, ids, teacher, T, w)
            continue
        # a gradient w T (q - p) of 2^57 or so: what is past 65504 by half a step is infinite in float16
        losses, bound, grad, bounds = R.distill(z, ids, teacher, T, w)
        got, got_grad = sc.distill_grad(z, ids, teacher, w, temperature=T)
        close(got, losses, bound, "losses")
        past, sure = grad.abs() >= 65520, (grad.abs() - 65520).abs() > bounds
        assert torch.equal(got_grad[past & sure].double(), grad[past & sure].sign() * math.inf)
        near = ~past & sure
        close(got_grad[near], grad[near], (bounds + rounding(dtype, grad))[near], "gradient")


@pytest.mark.parametrize("n,V", FORMS)
@pytest.mark.parametrize("far", [1e10, -1e10, 3e38, -3e38])
def test_logits_far_from_zero(n, V, far):
    g = gen(V)
    z = far * (1 - 3e-7 * randn(g, n, V).abs())  # a few steps of float32 apart
    z[::2] = torch.where(randn(g, *z[::2].shape) > 0, z[::2], randn(g, *z[::2].shape))
    ids, teacher = lists(g, z / 4, min(V, 9))
    check_distill(z, ids, randn(g, *ids.shape), 1.0, torch.rand(n, generator=g, device=DEV) + 0.1)
    check_balance(z, taken(g, z / 4, min(V, 3), wide=True), 64.0)


@pytest.mark.parametrize("n,V", FORMS)
@pytest.mark.parametrize("sign", [1, -1])
def test_the_magnitude_where_the_form_changes(n, V, sign):
    """Largest logits of lanes, waves and parts on both sides of m c = 2^20, c =
    log2(e) / T, and the next powers of two."""
    g = gen(V)
    for power in (19, 20, 21, 24):
        z = sign * 2.0 ** power / 1.4426950408889634 + randn(g, n, V) * 3
        z[1::3] += torch.linspace(-8, 8, V, device=DEV)  # whole waves on one side, others on the other
        z[2::3] -= torch.linspace(-8, 8, V, device=DEV)
        ids, teacher = lists(g, z, min(V, 9))
        check_distill(z, ids, teacher, 1.0, torch.rand(n, generator=g, device=DEV) + 0.1)
        check_balance(z, taken(g, z, min(V, 3), wide=True), 64.0)
    T = 10 * 1.4426950408889634 / 2 ** 20
    z = sign * (10 + 3e-5 * randn(g, n, V))
    ids, teacher = lists(g, z, min(V, 9))
    check_distill(z, ids, (sign * 10 + 3e-5 * randn(g, *ids.shape)), T, torch.rand(n, generator=g, device=DEV) + 0.1)


def test_rows_of_one_number():
    """Even weights, whatever the number."""
    for V in (3, 200, 1000, 1500, 16384, 16390, 40001):
        numbers = torch.tensor([0.0, 1.0, -1e5, 1e6, -1e9, 1e10, -1e20, 1e30, -3e38, 3e38], device=DEV)
        z = numbers[:, None].expand(-1, V).contiguous()
        ids = torch.zeros(len(numbers), 1, dtype=torch.int64, device=DEV)
        losses, grad = sc.distill_grad(z, ids, torch.zeros(len(numbers), 1, device=DEV))
        # two roundings of the sum's logarithm, at most 64 + 16 of the sum
        assert float((losses.double() - math.log(V)).abs().max()) <= R.depth(V) * 2.0 ** -23 * max(1.0, math.log(V))
        assert bool((grad[:, 1:].double() * V - 1).abs().max() <= (R.depth(V) + 8) * 2.0 ** -24)
