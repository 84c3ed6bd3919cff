"""Products of 8-bit rows are equal from call to call, with other work between the
calls and beside them on another stream."""
import pytest
import torch

import soft_clustering_amd as sc
from tests.test_gpu_losses import DEV, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,dim", [(4100, 4100, 1100), (300, 5000, 520), (65, 2048, 4096), (17, 5001, 1000), (1, 5001, 1000)])
def test_equal_from_call_to_call(m, n, dim, dtype):
    g = gen(m + n + dim)
    a, b = sc.byte_quantize(randn(g, m, dim)), sc.byte_quantize(randn(g, n, dim))
    other = sc.byte_quantize(randn(g, m, dim) * 1e3)
    first = sc.byte_product(a, b, dtype=dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    beside = []
    for i in range(8):
        sc.byte_product(other, b, dtype=dtype)
        with torch.cuda.stream(side):
            beside.append(sc.byte_product(a, b, dtype=dtype))
        assert torch.equal(sc.byte_product(a, b, dtype=dtype), first)
    side.synchronize()
    assert all(torch.equal(x, first) for x in beside)
