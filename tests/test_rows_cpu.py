"""The row operators without a GPU: the header and the binding agree, every
refusal comes before the device is touched, and the references that the GPU
tests use agree with hand-made cases."""
import ast
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import soft_clustering_amd as sc
from tests import rows_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, CAPACITY = 1, 6
P = ctypes.c_void_p(4096)     # aligned, never dereferenced: the call is refused first
ODD = ctypes.c_void_p(4097)


def test_header_binding_and_library_agree():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "flashgmm_rows.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gmm_[a-z_]+)\s*\(", src)))
    assert names == sorted(sc.ROW_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", sc.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r"\bT (gmm_[a-z_]+)$", out, flags=re.M))


def refused(status, text, want=INVALID):
    assert status == want, status
    assert text in sc.raw_library().gmm_last_error(None).decode()


def test_quantize_refusals():
    lib = sc.raw_library()
    good = dict(X=P, type=0, N=4, D=128, ldx=128, codes=P, ldc=64, scales=P, lds=4)

    def q(**kw):
        a = {**good, **kw}
        return lib.gmm_mx_quantize(a["X"], a["type"], a["N"], a["D"], a["ldx"], a["codes"], a["ldc"], a["scales"],
                                   a["lds"], None)

    refused(q(N=-1), "N must be")
    refused(q(N=(1 << 30) + 1), "N must be")
    refused(q(D=0), "D must be")
    refused(q(D=(1 << 20) + 1), "D must be")
    refused(q(type=3), "element type")
    refused(q(X=None), "X is NULL")
    refused(q(X=ODD), "aligned")
    refused(q(ldx=127), "row stride")
    refused(q(codes=None), "non-NULL")
    refused(q(scales=None), "non-NULL")
    refused(q(codes=ODD), "aligned")
    refused(q(scales=ODD), "aligned")
    refused(q(ldc=48), "code stride")
    refused(q(ldc=72), "code stride")
    refused(q(D=129, ldx=129), "code stride")
    refused(q(lds=6), "scale stride")
    assert q(N=0) == 0
    refused(lib.gmm_mx_dequantize(None, 64, P, 4, 4, 128, P, 0, 128, None), "non-NULL")
    refused(lib.gmm_mx_dequantize(P, 64, P, 4, 4, 128, P, 0, 127, None), "row stride")
    refused(lib.gmm_mx_dequantize(P, 64, P, 4, 4, 128, P, 5, 128, None), "element type")
    assert lib.gmm_mx_dequantize(P, 64, P, 4, 0, 128, P, 0, 128, None) == 0


def test_product_refusals():
    lib = sc.raw_library()
    good = dict(A=P, at=3, lda=64, as_=P, ldas=4, M=100, B=P, ldb=64, bs=P, ldbs=4, N=5, D=100, bias=None, C=P, ct=0,
                ldc=5, ws=None, wb=0)

    def q(**kw):
        a = {**good, **kw}
        return lib.gmm_mx_product(a["A"], a["at"], a["lda"], a["as_"], a["ldas"], a["M"], a["B"], a["ldb"], a["bs"],
                                  a["ldbs"], a["N"], a["D"], a["bias"], a["C"], a["ct"], a["ldc"], a["ws"], a["wb"],
                                  None)

    refused(q(M=-1), "M must be")
    refused(q(N=-1), "N must be")
    refused(q(D=0), "D must be")
    refused(q(at=4, lda=100), "element type")
    refused(q(A=None), "non-NULL")
    refused(q(as_=None), "non-NULL")
    refused(q(at=0, lda=99), "row stride")
    refused(q(bs=None), "B: codes")
    refused(q(ldb=60), "code stride")
    refused(q(ldbs=5), "scale stride")
    refused(q(ct=3), "C: unknown")
    refused(q(C=None), "C is NULL")
    refused(q(C=ODD), "aligned")
    refused(q(ldc=4), "row stride")
    refused(q(bias=ODD), "bias")
    assert q(M=0) == 0 and q(N=0) == 0
    need = lib.gmm_mx_product_workspace(0, 100, 5, 100)
    assert need > 0
    refused(q(at=0, lda=100), "workspace", CAPACITY)
    refused(q(at=0, lda=100, ws=P, wb=need - 1), "workspace", CAPACITY)
    refused(q(at=0, lda=100, ws=ctypes.c_void_p(4100), wb=need), "16-byte aligned")
    for bad in ((4, 1, 1, 1), (-1, 1, 1, 1), (0, -1, 1, 1), (0, 1, 1, 0)):
        assert lib.gmm_mx_product_workspace(*bad) == 0


def test_draw_refusals():
    lib = sc.raw_library()
    good = dict(z=P, type=0, N=4, V=10, ld=10, u=P, ts=None, t=1.0, ks=None, k=0, ps=None, p=1.0, ms=None, m=0.0,
                ids=P)

    def q(**kw):
        a = {**good, **kw}
        return lib.gmm_draw(a["z"], a["type"], a["N"], a["V"], a["ld"], a["u"], a["ts"], a["t"], a["ks"], a["k"],
                            a["ps"], a["p"], a["ms"], a["m"], a["ids"], None, 0, None)

    refused(q(N=-1), "N must be")
    refused(q(V=0), "V must be")
    refused(q(V=(1 << 20) + 1, ld=1 << 21), "V must be")
    refused(q(type=3), "element type")
    refused(q(z=None), "logits is NULL")
    refused(q(ld=9), "row stride")
    refused(q(t=-0.5), "temperature")
    refused(q(t=float("nan")), "temperature")
    refused(q(p=float("nan")), "top_p")
    refused(q(m=float("nan")), "min_p")
    refused(q(u=None), "non-NULL")
    refused(q(ids=None), "non-NULL")
    refused(q(ids=ODD), "aligned")
    refused(q(ts=ODD), "aligned")
    assert q(N=0) == 0


def test_binding_refusals_on_cpu_tensors():
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="GPU"):
        sc.mx_quantize(x)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        sc.mx_quantize(x.double())
    with pytest.raises(ValueError, match="2-D"):
        sc.mx_quantize(x[0])
    with pytest.raises(ValueError, match="GPU"):
        sc.draw(x, torch.zeros(4))
    c, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    rows = sc.MXRows(c, s, 100)
    assert len(rows) == 4 and len(rows[1:3]) == 2 and rows.nbytes == 4 * 68
    with pytest.raises(TypeError, match="slice"):
        rows[0]
    with pytest.raises(TypeError, match="slice"):
        rows[::2]
    with pytest.raises(ValueError, match="4 x 128|N x 128"):
        sc.MXRows(c, s, 129)
    with pytest.raises(TypeError, match="uint8"):
        sc.MXRows(c.int(), s, 128)
    with pytest.raises(ValueError, match="same rows"):
        sc.MXRows(c, s[:3], 128)
    with pytest.raises(ValueError, match="GPU"):
        sc.mx_product(rows, rows)
    with pytest.raises(ValueError, match="GPU"):
        sc.mx_dequantize(rows)
    with pytest.raises(TypeError, match="MXRows"):
        sc.mx_product(x, x)


def test_reference_quantize_by_hand():
    x = np.zeros((1, 64))
    # largest 7: e = 0; each midpoint goes to the even code; 7 saturates at 6
    x[0, :10] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.5]
    x[0, 32] = 2.0 ** -140
    x[0, 33] = -0.0
    codes, scales = R.quantize(x)
    v = R.values(codes, scales, 64)[0]
    assert v[:10].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -6]
    assert scales[0].tolist() == [127, 0, 0, 0]
    assert v[32] == 0 and np.signbit(v[33])
    x[0, 40] = np.inf
    codes, scales = R.quantize(x)
    assert scales[0, 1] == 255 and np.isnan(R.values(codes, scales, 64)[0, 32:]).all()


def test_reference_draw_by_hand():
    z = np.log([4.0, 1.0, 3.0, 2.0])  # weights 1, 1/4, 3/4, 1/2
    assert [R.draw(z, u) for u in (0.0, 0.39, 0.41, 0.49, 0.51, 0.79, 0.81, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert np.flatnonzero(R.kept(z, top_k=2)).tolist() == [0, 2]
    assert np.flatnonzero(R.kept(z, top_p=0.41)).tolist() == [0, 2]
    assert np.flatnonzero(R.kept(z, top_p=0.0)).tolist() == [0]
    assert np.flatnonzero(R.kept(z, top_k=3, top_p=0.8)).tolist() == [0, 2, 3]
    assert np.flatnonzero(R.kept(z, min_p=0.4)).tolist() == [0, 2, 3]
    assert np.flatnonzero(R.kept(np.zeros(6), top_k=4, top_p=0.5)).tolist() == [0, 1]
    assert R.draw([0.0, 5.0, 5.0], 0.9, temperature=0.0) == 1
    assert R.draw([-np.inf] * 3, 0.5) == -1 and R.draw([0.0, np.nan], 0.5) == -1 and R.draw([np.inf, 0], 0.5) == -1


def test_compressed_scan_refusals():
    from soft_clustering_amd import ivf_probe

    X = torch.arange(8 * 32, dtype=torch.float32).reshape(8, 32)
    rows = sc.MXRows(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8), 32)
    with pytest.raises(TypeError, match="MXRows"):
        ivf_probe.compressed_topk(X, X, X, 2, 4)
    with pytest.raises(ValueError, match="integer values"):
        ivf_probe.compressed_topk(X + 0.5, rows, X, 2, 4)
    with pytest.raises(ValueError, match="same width"):
        ivf_probe.compressed_topk(X[:, :31], rows, X, 2, 4)
    with pytest.raises(ValueError, match="same width"):
        ivf_probe.compressed_topk(X, rows[:7], X, 2, 4)
    for k, short in ((0, 4), (5, 4), (2, 9)):
        with pytest.raises(ValueError, match="shortlist"):
            ivf_probe.compressed_topk(X, rows, X, k, short)
    with pytest.raises(ValueError, match="on a GPU"):
        ivf_probe.compressed_topk(X, rows, X, 2, 4)


def test_draw_workspace_sizes():
    """The query at its smallest and largest arguments, no rows among them
    (in a child: it has to answer, not end the process)."""
    code = ("import soft_clustering_amd as sc; f = sc.raw_library().gmm_draw_workspace; "
            "print([[f(n, v) for v in (1, 16384, 16385, 131072, 1 << 20)] for n in (0, 1, 128, 129, 1 << 30)])")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.returncode
    none, one, most, more, all_ = ast.literal_eval(out.stdout.splitlines()[-1])
    assert none == more == all_ == [0] * 5
    assert one[:2] == most[:2] == [0, 0]
    assert one[2] == one[3] == one[4] > 0 and most[2:] == [128 * one[2]] * 3
    f = sc.raw_library().gmm_draw_workspace
    for bad in ((-1, 20000), ((1 << 30) + 1, 20000), (4, 0), (4, -5), (4, (1 << 20) + 1)):
        assert f(*bad) == 0


def test_widths_past_32_bits_are_refused():
    """The C ABI's widths are int32: a wider row must not be taken for a short one."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    from soft_clustering_amd.rows import _rows

    with FakeTensorMode():
        for width in (2 ** 31, 2 ** 32 + 5, 2 ** 40 + 128):
            x = torch.empty(1, width, dtype=torch.bfloat16, device="cuda")
            with pytest.raises(ValueError, match="rows of"):
                _rows(x, "logits")
        assert _rows(torch.empty(3, 2 ** 31 - 1, dtype=torch.bfloat16, device="cuda"), "X")[2] == 2 ** 31 - 1


def test_inputs_that_need_gradients_are_refused():
    """The products have no backward: a result without a graph would be a wrong
    gradient.  Without gradients (no_grad, detach) the same tensors are taken."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode():
        x = torch.empty(4, 128, device="cuda", requires_grad=True)
        plain = torch.empty(4, 128, device="cuda")
        rows = sc.MXRows(torch.empty(4, 64, dtype=torch.uint8, device="cuda"),
                         torch.empty(4, 4, dtype=torch.uint8, device="cuda"), 128)
        bias = torch.empty(4, device="cuda", requires_grad=True)
        with pytest.raises(ValueError, match="X requires"):
            sc.mx_quantize(x)
        with pytest.raises(ValueError, match="A requires"):
            sc.mx_product(x, rows)
        with pytest.raises(ValueError, match="bias requires"):
            sc.mx_product(plain, rows, bias=bias)
        with pytest.raises(ValueError, match="out requires"):
            sc.mx_dequantize(rows, out=x)
        with pytest.raises(ValueError, match="out requires"):
            sc.mx_product(rows, rows, out=torch.empty(4, 4, device="cuda", requires_grad=True))


def test_import_on_a_torch_without_gpu_support():
    """The package, its generators and the probe do not need torch's GPU bindings."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda')]: delattr(torch._C, n)\n"
            "import soft_clustering_amd as sc\n"
            "from soft_clustering_amd import datagen, ivf_probe\n"
            "X = torch.arange(12.0).reshape(4, 3)\n"
            "print(ivf_probe.exact_topk(X, X, 1)[0].flatten().tolist())\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert out.stdout.splitlines()[-1] == "[0, 1, 2, 3]"


def test_scan_bias():
    from soft_clustering_amd import ivf_probe

    g = torch.Generator().manual_seed(1)
    X = torch.randint(-300, 300, (5000, 37), generator=g).float()
    want = (X.double() ** 2).sum(1).div(-2).float()
    assert torch.equal(ivf_probe.scan_bias(X), want)
    assert torch.equal(ivf_probe.scan_bias(X, part=1000), want)   # parts of 27 rows
    assert torch.equal(ivf_probe.scan_bias(X, part=1), want)      # of one row
    assert ivf_probe.scan_bias(X[:0]).shape == (0,)
    X[4999, 36] += 0.5
    with pytest.raises(ValueError, match="integer values"):
        ivf_probe.scan_bias(X, part=1000)
    with pytest.raises(TypeError, match="float32"):
        ivf_probe.scan_bias(X.double())
    with pytest.raises(TypeError, match="MXRows"):
        ivf_probe.scan_bias([1.0])
    rows = sc.MXRows(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8), 37)
    for bad in (want[:7], want[:8].double(), want[:8, None]):
        with pytest.raises((TypeError, ValueError), match="bias"):
            ivf_probe.compressed_topk(X[:2], rows, X[:8], 2, 4, bias=bad)


def test_accuracy_of_the_weights():
    """The header promises weights within 1.2 * 2^-43 of the largest, V times that
    for a sum: half of a step of 2^-42 from rounding and the error of the
    polynomial of 2^f, |f| <= 1/2, which is found here from its constants (the
    weight is 2^n 2^f with n <= 0; the float64 operations add less than 2^-48)."""
    src = open(os.path.join(ROOT, "soft_clustering_amd", "csrc", "gmm_draw.hip")).read()
    body = src[src.index("double fixed_exp2("):]
    body = body[:body.index("return __hiloint2double")]
    c = [float.fromhex(v) for v in re.findall(r"0x1\.[0-9a-f]+p[+-]\d+", body)]
    assert len(c) == 9 and "q = fma(q, f, 1.0)" in body
    f = np.linspace(-0.5, 0.5, 400_001).astype(np.longdouble)
    q = np.zeros_like(f)
    for k in c + [1.0]:
        q = q * f + np.longdouble(k)
    worst = float(np.abs(q - np.exp2(f)).max())
    assert worst <= 2.0 ** -45.8
    assert 2.0 ** -43 + worst + 2.0 ** -48 <= 1.2 * 2.0 ** -43
    header = open(os.path.join(ROOT, "include", "flashgmm_rows.h")).read()
    assert "within 1.2 * 2^-43" in header


def test_sanitizer_exercise_covers_the_row_operators():
    """tests/native/rows_exercise.cpp calls every function of the header, and the
    host build under sanitizers holds every source of the library."""
    native = os.path.join(ROOT, "tests", "native")
    called = set(re.findall(r"\b(gmm_[a-z_]+)\s*\(", open(os.path.join(native, "rows_exercise.cpp")).read()))
    assert set(sc.ROW_EXPORTS) <= called
    script = open(os.path.join(native, "build_sanitized.sh")).read()
    sources = set(re.search(r"for src in ([a-z_ ]+); do", script).group(1).split())
    built = re.search(r"SOURCES = \[(.*?)\]", open(os.path.join(ROOT, "soft_clustering_amd", "build.py")).read(), re.S)
    assert sources == {v[:-4] for v in re.findall(r'"([a-z_]+\.hip)"', built.group(1))}
    assert "rows_exercise" in script


def test_memory_shared_by_a_result_and_an_input():
    """By brute force over the bytes of views of one buffer."""
    from soft_clustering_amd.rows import _overlap

    buf = torch.arange(60 * 20, dtype=torch.int16).reshape(60, 20)
    views = [buf[0:10, 0:5], buf[0:10, 5:9], buf[0:10, 4:9], buf[3:30, 18:20], buf[3:30, 0:20], buf[10:20, 0:5],
             buf[9, 0:5], buf[9, 6:20], buf[9:10, 5:20], buf[0:0], buf.view(-1)[7:1100], buf.view(30, 40)[2:9, 20:25],
             buf.view(30, 40)[2:9, 0:20], buf[2:3, 19:20], buf.view(-1)[9 * 20 + 5:9 * 20 + 17], buf[:, 7]]
    whole = [v for v in views if v.dim() == 2 or v.is_contiguous()]
    for a in whole:
        for b in whole:
            shared = bool(set(a.flatten().tolist()) & set(b.flatten().tolist()))
            found = _overlap(a, b)
            # never missed; views whose rows lie at different strides may be taken to overlap
            assert found or not shared, (a.shape, b.shape)
            same = a.shape[0] < 2 or b.shape[0] < 2 or a.stride(0) == b.stride(0) or a.dim() == 1 or b.dim() == 1
            assert found == shared or not same, (a.shape, b.shape)
