"""Distillation and balance without a GPU: every refusal comes before the device
is touched, and the references agree with torch's autograd."""
import ctypes
import math

import pytest
import torch

import soft_clustering_amd as sc
from tests import losses_reference as R

INVALID, CAPACITY = 1, 6
P = ctypes.c_void_p(4096)     # aligned, never dereferenced: the call is refused first
ODD = ctypes.c_void_p(4097)


def refused(status, text, want=INVALID):
    assert status == want, status
    assert text in sc.raw_library().gmm_last_error(None).decode()


def test_distill_refusals():
    lib = sc.raw_library()
    good = dict(z=P, type=0, N=4, V=10, ld=10, ids=P, bits=32, ldi=3, t=P, tt=0, ldt=3, k=3, T=1.0)

    def inputs(kw):
        a = {**good, **kw}
        return [a[n] for n in ("z", "type", "N", "V", "ld", "ids", "bits", "ldi", "t", "tt", "ldt", "k", "T")]

    def forward(losses=P, stats=None, weights=None, grad=None, ldg=10, **kw):
        return lib.gmm_distill(*inputs(kw), losses, stats, weights, 1.0, grad, ldg, None, 0, None)

    def backward(stats=P, weights=P, ldw=1, grad=P, ldg=10, **kw):
        return lib.gmm_distill_backward(*inputs(kw), stats, weights, ldw, grad, ldg, None)

    for call in (forward, backward):
        refused(call(N=-1), "N must be")
        refused(call(N=(1 << 30) + 1), "N must be")
        refused(call(V=0), "V must be")
        refused(call(V=(1 << 20) + 1), "V must be")
        refused(call(type=3), "logits: unknown element type")
        refused(call(z=None), "logits is NULL")
        refused(call(z=ODD), "aligned")
        refused(call(ld=9), "row stride")
        for bits in (0, 16, 33):
            refused(call(bits=bits), "id_bits")
        for k in (0, -1, 1025):
            refused(call(k=k, ldi=2000, ldt=2000), "k must be")
        refused(call(ids=None), "ids is NULL")
        refused(call(ids=ctypes.c_void_p(4100), bits=64), "aligned")
        refused(call(ldi=2), "ids: row stride")
        refused(call(t=None), "teacher is NULL")
        refused(call(tt=4), "teacher: unknown element type")
        refused(call(ldt=2), "teacher: row stride")
        for T in (0.0, -1.0, float("nan"), float("inf"), 1e-30, 1e30):
            refused(call(T=T), "temperature")
        refused(call(grad=ODD), "aligned")
        refused(call(grad=P, ldg=9), "grad: row stride")
        assert call(N=0) == 0
    refused(forward(losses=None), "losses is NULL")
    refused(forward(stats=ODD), "aligned")
    refused(forward(weights=ODD), "aligned")
    refused(backward(grad=None), "grad is NULL")
    refused(backward(stats=None), "non-NULL")
    refused(backward(weights=None), "non-NULL")
    refused(backward(weights=ODD), "aligned")
    refused(backward(ldw=-1), "stride")
    for bad in ((-1, 4, 1), (1, 0, 1), (1, (1 << 20) + 1, 1), (1, 4, 0), (1, 4, 1025), ((1 << 30) + 1, 4, 1)):
        assert lib.gmm_distill_workspace(*bad) == 0


def test_balance_refusals():
    lib = sc.raw_library()
    good = dict(z=P, type=0, N=4, K=10, ld=10, ids=P, bits=32, ldi=2, k=2, counts=P, loss=P, stats=P, grad=None, ldg=10,
                ws=P, wb=1 << 30)

    def forward(**kw):
        a = {**good, **kw}
        return lib.gmm_balance(a["z"], a["type"], a["N"], a["K"], a["ld"], a["ids"], a["bits"], a["ldi"], a["k"],
                               a["counts"], a["loss"], a["stats"], 1.0, a["grad"], a["ldg"], a["ws"], a["wb"], None)

    refused(forward(N=-1), "N must be")
    refused(forward(K=0), "K must be")
    refused(forward(K=(1 << 20) + 1), "K must be")
    refused(forward(type=4), "element type")
    refused(forward(z=None), "logits is NULL")
    refused(forward(ld=9), "row stride")
    refused(forward(bits=8), "id_bits")
    refused(forward(k=0), "k must be")
    refused(forward(k=1025, ldi=2000), "k must be")
    refused(forward(ids=None), "ids is NULL")
    refused(forward(ids=ODD), "aligned")
    refused(forward(ldi=1), "ids: row stride")
    refused(forward(counts=None), "non-NULL")
    refused(forward(loss=None), "non-NULL")
    refused(forward(stats=None), "non-NULL")
    refused(forward(counts=ctypes.c_void_p(4100)), "aligned")
    refused(forward(stats=ODD), "aligned")
    refused(forward(grad=P, ldg=9), "grad: row stride")
    need = lib.gmm_balance_workspace(4, 10, 2)
    assert need > 0
    refused(forward(wb=need - 1), "workspace", CAPACITY)
    refused(forward(ws=None), "workspace", CAPACITY)
    refused(forward(ws=ctypes.c_void_p(4104)), "16-byte aligned")

    def backward(z=P, type=0, N=4, K=10, ld=10, stats=P, weight=P, grad=P, ldg=10):
        return lib.gmm_balance_backward(z, type, N, K, ld, stats, weight, grad, ldg, None)

    refused(backward(N=-1), "N must be")
    refused(backward(type=7), "element type")
    refused(backward(z=None), "logits is NULL")
    refused(backward(ld=9), "row stride")
    refused(backward(grad=None), "grad is NULL")
    refused(backward(ldg=9), "grad: row stride")
    refused(backward(stats=None), "non-NULL")
    refused(backward(weight=ODD), "aligned")
    assert backward(N=0) == 0
    assert lib.gmm_balance_stats(-1, 4) == lib.gmm_balance_stats(4, 0) == lib.gmm_balance_stats(4, (1 << 20) + 1) == 0
    for bad in ((-1, 4, 1), (1, 0, 1), (1, 4, 0), (1, 4, 1025), (1, (1 << 20) + 1, 1)):
        assert lib.gmm_balance_workspace(*bad) == 0
    for N in (0, 1, 1000, 1 << 30):  # bounded whatever the sizes, and queries that answer
        for K in (1, 16384, 65537, 1 << 20):
            for k in (1, 1024):
                assert 0 < lib.gmm_balance_workspace(N, K, k) <= (1 << 25) + (1 << 18)


def test_binding_refusals():
    z, ids, t = torch.zeros(4, 10), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: sc.distill(z, ids, t), lambda: sc.distill_grad(z, ids, t), lambda: sc.balance(z, ids),
                 lambda: sc.balance_grad(z, ids)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        sc.distill(z.double(), ids, t)
    with pytest.raises(TypeError, match="torch.Tensor"):
        sc.balance([1.0], ids)


def test_binding_refusals_on_gpu_tensors():
    """On fake tensors: nothing is launched."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode():
        def f(*shape, **kw):
            return torch.empty(*shape, device="cuda", **kw)

        z, ids, t = f(4, 10), f(4, 2, dtype=torch.int32), f(4, 2)
        for fn in (sc.distill, sc.distill_grad):
            with pytest.raises(TypeError, match="int32 or int64"):
                fn(z, ids.float(), t)
            with pytest.raises(ValueError, match="4 rows"):
                fn(z, f(3, 2, dtype=torch.int64), t)
            with pytest.raises(ValueError, match="4 rows"):
                fn(z, f(4, dtype=torch.int64), t)
            with pytest.raises(ValueError, match="between 1 and 1024"):
                fn(z, f(4, 0, dtype=torch.int64), f(4, 0))
            with pytest.raises(ValueError, match="between 1 and 1024"):
                fn(z, f(4, 1025, dtype=torch.int64), f(4, 1025))
            with pytest.raises(ValueError, match="contiguous"):
                fn(z, f(2, 4, dtype=torch.int32).t(), t)
            with pytest.raises(ValueError, match="overlap"):
                fn(z, f(1, 2, dtype=torch.int32).expand(4, 2), t)
            with pytest.raises(ValueError, match="4 x 2"):
                fn(z, ids, f(4, 3))
            with pytest.raises(ValueError, match="teacher requires"):
                fn(z, ids, f(4, 2, requires_grad=True))
        leaf = f(4, 10, requires_grad=True)
        with pytest.raises(ValueError, match="logits requires"):
            sc.distill_grad(leaf, ids, t)
        with pytest.raises(ValueError, match="logits requires"):
            sc.balance_grad(leaf, ids)
        with pytest.raises(TypeError, match="weights must be"):
            sc.distill_grad(z, ids, t, f(4, dtype=torch.float64))
        with pytest.raises(ValueError, match="weights must be"):
            sc.distill_grad(z, ids, t, f(3))
        with pytest.raises(ValueError, match="shape"):
            sc.distill_grad(z, ids, t, out=f(4, 9))
        with pytest.raises(TypeError, match="out must be"):
            sc.balance_grad(z, ids, out=f(4, 10, dtype=torch.bfloat16))
        with pytest.raises(ValueError, match="out requires"):
            sc.balance_grad(z, ids, out=leaf)


def test_references_against_autograd():
    g = torch.Generator().manual_seed(1)
    z = torch.randn(6, 12, generator=g, dtype=torch.float64, requires_grad=True)
    t = torch.randn(6, 4, generator=g, dtype=torch.float64)
    ids = torch.randint(0, 12, (6, 4), generator=g)
    ids[1, 2:], ids[2] = -1, -1
    w = torch.rand(6, generator=g)
    T = 1.7
    p = torch.softmax((t / T).masked_fill(ids < 0, -math.inf), 1).nan_to_num(0.0)
    logq = torch.log_softmax(z / T, 1).gather(1, ids.clamp(min=0))
    losses = T * T * (torch.special.xlogy(p, p) - p * logq).sum(1)
    grad, = torch.autograd.grad((losses * w).sum(), z)
    got = R.distill(z.detach(), ids, t, T, w)
    # T is rounded to float32 in the reference
    assert torch.allclose(got[0], losses.detach(), atol=1e-6) and torch.allclose(got[2], grad, atol=1e-6)
    assert float(got[0][2]) == 0 and not bool(got[2][2].any())

    ids[0] = -1
    counted = (ids >= 0).any(1)
    counts = torch.bincount(ids[ids >= 0], minlength=12).double()
    mean = (torch.softmax(z, 1) * counted[:, None]).sum(0) / counted.sum()
    loss = 12 * (counts / counts.sum() * mean).sum()
    grad, = torch.autograd.grad(loss * 0.3, z)
    got = R.balance(z.detach(), ids, 0.3)
    assert torch.allclose(got[0], loss.detach()) and torch.allclose(got[3], grad)
    assert torch.equal(got[2], counts.long())


def test_workspace_of_no_rows():
    """Of any width, none: also where rows would be divided."""
    from soft_clustering_amd import rows

    for width in (1, 1000, 16385, 40000, 131072, 2 ** 20):
        assert rows._lib.gmm_distill_workspace(0, width, 5) == 0
        assert rows._lib.gmm_balance_stats(0, width) >= width
        assert rows._lib.gmm_balance_workspace(0, width, 5) > 0
