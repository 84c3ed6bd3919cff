"""Components with the same logit (and as many of a row's ids) have the same
gradient to the last bit, wherever in the row they lie: a row's numbers are the
same in all lanes that form its gradient, and where lanes write the same element
(vectors at a row's end are placed over each other) they write the same.  Rows
held by several waves are not meant: a wave's exponentials are rounded from its
own largest logit, and each element has one owner there."""
import pytest
import torch

import soft_clustering_amd as sc
from tests.test_gpu_losses import DEV, NAMES, TYPES, gen, randn

pytestmark = pytest.mark.gpu


def few_values(g, n, V, dtype):
    """(logits that take 8 values, which of them)."""
    at = torch.randint(0, 8, (n, V), generator=g, device=DEV)
    return (randn(g, n, 8) * 2).to(dtype).gather(1, at), at


def check_equal(grad, at, free):
    for v in range(8):
        there = (at == v) & free
        high = grad.float().masked_fill(~there, -float("inf")).amax(1)
        low = grad.float().masked_fill(~there, float("inf")).amin(1)
        some = there.any(1)
        assert torch.equal(high[some], low[some]), v


# 16 lanes, a wave, whole long rows (held, and read again behind what is held), divided rows
@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,V", [(500, 203), (500, 1001), (300, 32771), (260, 140003), (5, 40007), (200, 70001)])
def test_distill(n, V, dtype):
    g = gen(n + V)
    z, at = few_values(g, n, V, dtype)
    ids = torch.randint(0, V, (n, 7), generator=g, device=DEV)
    free = torch.ones(n, V, dtype=torch.bool, device=DEV).scatter_(1, ids, False)
    teacher, w = randn(g, n, 7).to(dtype), torch.rand(n, generator=g, device=DEV) + 0.5
    check_equal(sc.distill_grad(z, ids, teacher, w, temperature=1.3)[1], at, free)
    leaf = z.detach().requires_grad_()
    check_equal(torch.autograd.grad(sc.distill(leaf, ids, teacher, 1.3), leaf, w)[0], at, free)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,K", [(40, 203), (500, 203), (500, 1001), (300, 16389), (200, 70001)])
def test_balance(n, K, dtype):
    g = gen(n + 3 * K)
    z, at = few_values(g, n, K, dtype)
    ids = torch.randint(0, 5, (n, 2), generator=g, device=DEV)
    free = (torch.arange(K, device=DEV) >= 5).expand(n, K)  # counted by none
    check_equal(sc.balance_grad(z, ids, 1000.0)[2], at, free)
    leaf = z.detach().requires_grad_()
    check_equal(torch.autograd.grad(1000.0 * sc.balance(leaf, ids)[0], leaf)[0], at, free)
