"""The balance's gradient in every form of its kernels: rows that take no component
have gradient 0, whatever their logits and the loss's weight; an id out of range
makes the whole gradient NaN, theirs included."""
import pytest
import torch

import soft_clustering_amd as sc
from tests import losses_reference as R
from tests.test_gpu_losses import DEV, NAMES, TYPES, close, gen, randn, rounding, taken

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

# shorter than a vector, 16 lanes, a wave, 4 and 16 waves, long rows; alone in one workgroup and not
FORMS = [(30, 3), (30, 64), (300, 64), (30, 700), (300, 700), (30, 1500), (30, 5000), (30, 20000)]


def gradients(z, ids, weight):
    yield "in one pass", sc.balance_grad(z, ids, weight)[2]
    leaf = z.detach().requires_grad_()
    loss, _ = sc.balance(leaf, ids)
    yield "by autograd", torch.autograd.grad(loss, leaf, torch.tensor(weight, device=DEV))[0]


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,K", FORMS)
def test_rows_that_take_nothing(n, K, dtype):
    g = gen(K)
    z = (randn(g, n, K) * 2).to(dtype)
    ids = taken(g, z, 2, True)
    ids[:5] = -1
    ids[5:, 0] = 0  # the others take one
    ref = z.clone()
    z[0, K - 1], z[1, 0], z[2], z[3] = INF, NAN, -INF, INF
    _, _, counts, want, bounds = R.balance(ref, ids, 8.0)
    for way, grad in gradients(z, ids, 8.0):
        close(grad, want, bounds + rounding(dtype, want), way)
        assert not bool(grad[:5].any()), way
    for weight in (INF, NAN):
        for way, grad in gradients(z, ids, weight):
            assert not bool(grad[:5].any()), (way, weight)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n,K", FORMS)
def test_an_id_out_of_range(n, K, dtype):
    g = gen(K + 1)
    z = (randn(g, n, K) * 2).to(dtype)
    ids = taken(g, z, 2, True)
    ids[:5] = -1
    for bad in (K, 2 ** 31 - 1, 2 ** 40):
        ids[n - 1, 1] = bad
        for weight in (8.0, 0.0):
            for way, grad in gradients(z, ids, weight):
                assert bool(torch.isnan(grad).all()), (way, bad, weight)
