"""One row of A against rows of B: a result goes by the two rows alone, to the last
bit, wherever the row of B lies."""
import pytest
import torch

import soft_clustering_amd as sc
from tests.test_gpu_losses import DEV, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [1000, 1024, 2000, 4096, 5000, 9001])  # 1, 2 and 4 steps at once, and several times
def test_equal_rows_have_equal_results(dim):
    g = gen(dim)
    a, b = randn(g, 1, dim), randn(g, 40, dim)
    same = sc.byte_quantize(b[:1].repeat(1001, 1))
    got = sc.byte_product(a, same)
    assert bool((got == got[0, 0]).all())
    rows = sc.byte_quantize(b)
    whole = sc.byte_product(a, rows)
    for s in range(1, 9):
        assert torch.equal(sc.byte_product(a, rows[s:]), whole[:, s:])
        assert torch.equal(sc.byte_product(sc.byte_quantize(a), rows[s:]), whole[:, s:])
