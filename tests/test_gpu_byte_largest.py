"""The largest numbers in 8-bit rows: float32's largest are rounded to 2^128, which is
infinite as a float32 value and, with float32 and float16 results, in products; what is
rounded below stays a number."""
import pytest
import torch

import soft_clustering_amd as sc
from tests.test_gpu_losses import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [100, 1024])
@pytest.mark.parametrize("m", [1, 5, 40, 70, 300])
def test_largest_numbers(m, dim):
    top = torch.finfo(torch.float32).max
    b = torch.zeros(70, dim, device=DEV)
    b[0], b[1], b[2] = top, -top, 1.9 * 2.0 ** 126  # the last to 1.875 * 2^126
    rows = sc.byte_quantize(b)
    values = sc.byte_dequantize(rows)
    assert bool((values[0] == float("inf")).all()) and bool((values[1] == -float("inf")).all())
    assert bool((values[2] == 1.875 * 2.0 ** 126).all())
    a = torch.full((m, dim), 2.0 ** -120, device=DEV)
    for dtype in (torch.float32, torch.float16):
        got = sc.byte_product(a, rows, dtype=dtype)
        assert bool((got[:, 0] == float("inf")).all()) and bool((got[:, 1] == -float("inf")).all())
        sums = torch.full((m,), dim * 1.875 * 2.0 ** 6, device=DEV)  # 122880 of 1024 values: infinite in float16
        assert torch.equal(got[:, 2], sums.to(dtype))
        assert not bool(got[:, 3:].any())
    got = sc.byte_product(a, rows, dtype=torch.bfloat16)  # there it may be its value
    assert bool(((got[:, 0] == float("inf")) | (got[:, 0] == dim * 256)).all()) and not bool(got[:, 3:].any())
