"""Rows in 8 bits without a GPU: every refusal comes before the device is
touched, and the reference that the GPU tests use agrees with hand-made cases."""
import ctypes

import numpy as np
import pytest
import torch

import soft_clustering_amd as sc
from tests import byte_reference as R

INVALID, CAPACITY = 1, 6
P = ctypes.c_void_p(4096)     # aligned, never dereferenced: the call is refused first
ODD = ctypes.c_void_p(4097)


def refused(status, text, want=INVALID):
    assert status == want, status
    assert text in sc.raw_library().gmm_last_error(None).decode()


def test_quantize_refusals():
    lib = sc.raw_library()
    good = dict(X=P, type=0, N=4, D=128, ldx=128, codes=P, ldc=128, scales=P, lds=4)

    def q(**kw):
        a = {**good, **kw}
        return lib.gmm_byte_quantize(a["X"], a["type"], a["N"], a["D"], a["ldx"], a["codes"], a["ldc"], a["scales"],
                                     a["lds"], None)

    refused(q(N=-1), "N must be")
    refused(q(N=(1 << 30) + 1), "N must be")
    refused(q(D=0), "D must be")
    refused(q(D=(1 << 20) + 1), "D must be")
    for t in (-1, 3, 4):
        refused(q(type=t), "element type")
    refused(q(X=None), "X is NULL")
    refused(q(X=ODD), "aligned")
    refused(q(ldx=127), "row stride")
    refused(q(codes=None), "non-NULL")
    refused(q(scales=None), "non-NULL")
    refused(q(codes=ctypes.c_void_p(4104)), "aligned")
    refused(q(scales=ctypes.c_void_p(4098)), "aligned")
    refused(q(ldc=112), "code stride")
    refused(q(ldc=136), "code stride")
    refused(q(ldc=(1 << 23) + 16), "code stride")
    refused(q(D=129, ldx=129), "code stride")
    refused(q(lds=6), "scale stride")
    refused(q(D=513, ldx=513, ldc=640), "scale stride")  # five groups: 8 scale bytes
    assert q(N=0) == 0
    refused(lib.gmm_byte_dequantize(None, 128, P, 4, 4, 128, P, 0, 128, None), "non-NULL")
    refused(lib.gmm_byte_dequantize(P, 128, P, 4, 4, 128, P, 0, 127, None), "row stride")
    refused(lib.gmm_byte_dequantize(P, 128, P, 4, 4, 128, P, 5, 128, None), "element type")
    refused(lib.gmm_byte_dequantize(P, 128, P, 4, 4, 128, None, 0, 128, None), "X is NULL")
    assert lib.gmm_byte_dequantize(P, 128, P, 4, 0, 128, P, 0, 128, None) == 0


def test_product_refusals():
    lib = sc.raw_library()
    good = dict(A=P, at=4, lda=128, as_=P, ldas=4, M=100, B=P, ldb=128, bs=P, ldbs=4, N=5, D=100, bias=None, C=P, ct=0,
                ldc=5, ws=None, wb=0)

    def q(**kw):
        a = {**good, **kw}
        return lib.gmm_byte_product(a["A"], a["at"], a["lda"], a["as_"], a["ldas"], a["M"], a["B"], a["ldb"], a["bs"],
                                    a["ldbs"], a["N"], a["D"], a["bias"], a["C"], a["ct"], a["ldc"], a["ws"], a["wb"],
                                    None)

    refused(q(M=-1), "M must be")
    refused(q(N=-1), "N must be")
    refused(q(D=0), "D must be")
    refused(q(at=3, lda=100), "element type")  # 4-bit rows are not mixed with 8-bit ones
    refused(q(A=None), "non-NULL")
    refused(q(as_=None), "non-NULL")
    refused(q(at=0, lda=99), "row stride")
    refused(q(bs=None), "B: codes")
    refused(q(ldb=120), "code stride")
    refused(q(ldbs=5), "scale stride")
    refused(q(ct=4), "C: unknown")
    refused(q(C=None), "C is NULL")
    refused(q(C=ODD), "aligned")
    refused(q(ldc=4), "row stride")
    refused(q(bias=ODD), "bias")
    assert q(M=0) == 0 and q(N=0) == 0
    need = lib.gmm_byte_product_workspace(0, 100, 5, 100)
    assert need >= 100 * 132
    refused(q(at=0, lda=100), "workspace", CAPACITY)
    refused(q(at=0, lda=100, ws=P, wb=need - 1), "workspace", CAPACITY)
    refused(q(at=0, lda=100, ws=ctypes.c_void_p(4100), wb=need), "16-byte aligned")
    assert lib.gmm_byte_product_workspace(4, 100, 5, 100) == 0
    for bad in ((3, 1, 1, 1), (5, 1, 1, 1), (-1, 1, 1, 1), (0, -1, 1, 1), (0, 1, 1, 0), (0, 1, 1, (1 << 20) + 1)):
        assert lib.gmm_byte_product_workspace(*bad) == 0


def test_binding_refusals_on_cpu_tensors():
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="GPU"):
        sc.byte_quantize(x)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        sc.byte_quantize(x.double())
    c, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    rows = sc.ByteRows(c, s, 100)
    assert len(rows) == 4 and len(rows[1:3]) == 2 and rows.nbytes == 4 * 132
    assert isinstance(rows[1:3], sc.ByteRows) and rows[1:3].codes.data_ptr() == c[1:].data_ptr()
    with pytest.raises(TypeError, match="slice"):
        rows[0]
    with pytest.raises(ValueError, match="N x 256"):
        sc.ByteRows(c, s, 129)
    with pytest.raises(TypeError, match="uint8"):
        sc.ByteRows(c.int(), s, 128)
    with pytest.raises(ValueError, match="same rows"):
        sc.ByteRows(c, s[:3], 128)
    with pytest.raises(ValueError, match="multiple of 16"):
        sc.ByteRows(torch.zeros(4, 136, dtype=torch.uint8)[:, :128], s, 128)
    with pytest.raises(ValueError, match="GPU"):
        sc.byte_product(rows, rows)
    with pytest.raises(ValueError, match="GPU"):
        sc.byte_dequantize(rows)
    four = sc.MXRows(c[:, :64], s, 128)
    for call in (lambda: sc.byte_product(x, four), lambda: sc.byte_dequantize(four), lambda: sc.byte_product(x, x)):
        with pytest.raises(TypeError, match="ByteRows"):
            call()
    with pytest.raises(TypeError, match="MXRows"):
        sc.mx_product(x, rows)


def test_rows_that_need_gradients_are_refused():
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode():
        x = torch.empty(4, 128, device="cuda", requires_grad=True)
        rows = sc.ByteRows(torch.empty(4, 128, dtype=torch.uint8, device="cuda"),
                           torch.empty(4, 4, dtype=torch.uint8, device="cuda"), 128)
        with pytest.raises(ValueError, match="X requires"):
            sc.byte_quantize(x)
        with pytest.raises(ValueError, match="A requires"):
            sc.byte_product(x, rows)
        with pytest.raises(ValueError, match="out requires"):
            sc.byte_dequantize(rows, out=x)
        with pytest.raises(TypeError, match="MXRows"):
            sc.mx_product(rows, rows)


def test_reference_quantize_by_hand():
    assert R.GRID[[1, 8, 126]].tolist() == [2.0 ** -9, 2.0 ** -6, 448.0]
    x = np.zeros((1, 256))
    # largest 448: e = 0; midpoints go to the even code
    x[0, :8] = [448, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, -0.0, -(2.0 ** -11), 440]
    x[0, 128:130] = 449, 1
    codes, scales = R.quantize(x)
    v = R.values(codes, scales, 256)[0]
    assert v[:8].tolist() == [448, 16, 20, 0, 2.0 ** -8, 0, 0, 448] and np.signbit(v[[5, 6]]).all()
    assert scales[0].tolist() == [127, 128, 0, 0] and v[128:130].tolist() == [448, 1]
    x[0, 3] = np.nan
    codes, scales = R.quantize(x)
    assert scales[0, 0] == 255 and np.isnan(R.values(codes, scales, 256)[0, :128]).all()
    tiny = np.zeros((1, 5))
    tiny[0] = [2.0 ** -119, 2.0 ** -136, 2.0 ** -137, 3 * 2.0 ** -137, 2.0 ** -149]
    codes, scales = R.quantize(tiny)
    assert scales[0, 0] == 0
    assert R.values(codes, scales, 5)[0].tolist() == [2.0 ** -119, 2.0 ** -136, 0, 2.0 ** -135, 0]


def test_reference_agrees_with_torch():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 384, generator=g) * torch.exp(2 * torch.randn(40, 1, generator=g))
    codes, scales = R.quantize(x.numpy())
    e = torch.from_numpy(scales.astype(np.int32))[:, :3] - 127
    want = torch.ldexp(x.view(40, 3, 128), -e[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(40, -1)
    assert np.array_equal(codes, want.numpy())
