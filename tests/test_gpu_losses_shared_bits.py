"""Distillation where listed ids share a bit of the kernels' record of ids seen:
different ids a multiple of its length apart, some of them listed twice as well.
Only rows longer than the record have such ids: whole rows of one workgroup, and
divided ones whose parts are longer."""
import os
import re

import pytest
import torch

from tests.test_gpu_losses import DEV, check_distill, gen, randn

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(os.path.dirname(__file__), "..", "soft_clustering_amd", "csrc", "gmm_losses.hip")
BITS = int(re.search(r"constexpr int kSeenBits = (\d+);", open(SOURCE).read()).group(1))


@pytest.mark.parametrize("n,V,k", [(256, 2 * BITS + 6, 1024), (257, 3 * BITS - 1, 70), (200, 8 * BITS, 1024),
                                   (250, 8 * BITS - 3, 100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ids_that_share_bits(n, V, k, dtype):
    assert V <= 1 << 20
    g = gen(n + V)
    z = randn(g, n, V).to(dtype)
    near = torch.randint(0, k // 4, (n, k), generator=g, device=DEV)  # some 4 places to a bit
    far = torch.randint(0, -(-V // BITS), (n, k), generator=g, device=DEV)
    ids = near * 37 + far * BITS
    ids = torch.where(ids < V, ids, near)
    ids[:, k // 2] = -1
    for row in range(0, n, 50):  # different ids of a row do share bits, and there are repeated ones
        own = ids[row][ids[row] >= 0]
        assert len((own.unique() % BITS).unique()) < len(own.unique()) < len(own)
    check_distill(z, ids, randn(g, n, k).to(dtype), 1.0, torch.ones(n, device=DEV))
