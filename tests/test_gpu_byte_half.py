"""float16 results of products of 8-bit rows: sums in float32, whatever the number
of rows.  A result that is small against its terms keeps what a sum cut below a
part of the largest term would lose."""
import pytest
import torch

import soft_clustering_amd as sc
from tests.test_gpu_losses import DEV, close, gen, randn, rounding

pytestmark = pytest.mark.gpu
M = [1, 17, 64, 65, 300, 1000]


@pytest.mark.parametrize("m", M)
@pytest.mark.parametrize("dim", [16, 128, 1000])
def test_terms_that_cancel(m, dim):
    """256 - 256 + 7 2^-6, 2^-6 being 2^-14 of 256: every partial sum is exact in float32
    (multiples of 2^-6 up to 2^9)."""
    a = torch.ones(m, dim, device=DEV)
    b = torch.zeros(300, dim, device=DEV)
    a[:, 1:8] = 2.0 ** -3
    b[:, 1:8] = 2.0 ** -3
    b[:, 0], b[:, 8] = 256, -256
    rows = sc.byte_quantize(b)
    assert torch.equal(sc.byte_dequantize(rows), b)
    for lhs in (a, sc.byte_quantize(a)):
        got = sc.byte_product(lhs, rows, dtype=torch.float16)
        assert bool((got == 7 * 2.0 ** -6).all())


@pytest.mark.parametrize("m", M)
@pytest.mark.parametrize("n,dim", [(300, 100), (1001, 777), (300, 4096)])
def test_against_float64(m, n, dim):
    g = gen(m + n + dim)
    a, b = sc.byte_quantize(randn(g, m, dim)), sc.byte_quantize(randn(g, n, dim) / dim ** 0.5)
    b.scales[0].clamp_(max=100)  # a row of small values
    x, y = sc.byte_dequantize(a).double(), sc.byte_dequantize(b).double()
    want, size = x @ y.T.contiguous(), x.abs() @ y.abs().T.contiguous()
    # products are exact; a float32 sum of dim terms is off by dim 2^-24 of their magnitudes at most
    close(sc.byte_product(a, b, dtype=torch.float16), want, rounding(torch.float16, want) + dim * 2.0 ** -24 * size * 1.001,
          f"{m} x {n} x {dim}")


def test_results_do_not_depend_on_the_rows_beside_them():
    """A row's results are those of float32 sums in any batch: the differences are those of
    two orders of the sum, before one rounding to float16."""
    g = gen(5)
    a, b = sc.byte_quantize(randn(g, 300, 500)), sc.byte_quantize(randn(g, 400, 500))
    size = sc.byte_dequantize(a).abs().double() @ sc.byte_dequantize(b).abs().double().T.contiguous()
    whole, part = sc.byte_product(a, b, dtype=torch.float16).double(), sc.byte_product(a[:20], b, dtype=torch.float16).double()
    assert bool(((whole[:20] - part).abs() <= 500 * 2.0 ** -23 * size[:20] + 2.0 ** -10 * part.abs()).all())
