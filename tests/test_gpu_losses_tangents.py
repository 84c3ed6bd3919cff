"""A tangent of the losses' weights in the backward pass (forward over reverse) is
refused: the gradient would come back without it."""
import pytest
import torch
from torch.autograd import forward_ad

import soft_clustering_amd as sc
from tests.test_gpu_losses import DEV, gen, randn

pytestmark = pytest.mark.gpu


def test_tangents_of_the_weights():
    g = gen(1)
    leaf = randn(g, 6, 50).requires_grad_()
    ids = torch.randint(0, 50, (6, 3), generator=g, device=DEV)
    losses, loss = sc.distill(leaf, ids, randn(g, 6, 3)), sc.balance(leaf, ids)[0]
    for out in (losses, loss):
        one = torch.ones_like(out)
        with forward_ad.dual_level():
            with pytest.raises(ValueError, match="tangent"):
                torch.autograd.grad(out, leaf, forward_ad.make_dual(one, one), retain_graph=True)
        assert bool(torch.isfinite(torch.autograd.grad(out, leaf, one)[0]).all())
