"""Tensors with a forward-mode tangent are refused wherever a result would lose it,
on fake tensors: nothing is launched."""
import pytest
import torch
from torch.autograd import forward_ad

import soft_clustering_amd as sc


@pytest.fixture
def f():
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode(), forward_ad.dual_level():
        def make(*shape, dual=False, **kw):
            t = torch.empty(*shape, device="cuda", **kw)
            return forward_ad.make_dual(t, torch.empty_like(t)) if dual else t

        yield make


def refused(name, fn, *args, **kw):
    with pytest.raises(ValueError, match=f"{name} has a forward-mode tangent"):
        fn(*args, **kw)


def test_losses(f):
    z, ids, t = f(4, 10), f(4, 2, dtype=torch.int32), f(4, 2)
    dual, leaf = f(4, 10, dual=True), forward_ad.make_dual(f(4, 10, requires_grad=True), f(4, 10))
    assert not dual.requires_grad and leaf.requires_grad
    for logits in (dual, leaf):
        refused("logits", sc.distill, logits, ids, t)
        refused("logits", sc.distill_grad, logits, ids, t)
        refused("logits", sc.balance, logits, ids)
        refused("logits", sc.balance_grad, logits, ids)
        with torch.no_grad():  # off for backward graphs, not for tangents
            refused("logits", sc.distill, logits, ids, t)
            refused("logits", sc.balance, logits, ids)
    for fn in (sc.distill, sc.distill_grad):
        refused("teacher", fn, z, ids, f(4, 2, dual=True))
        refused("teacher", fn, f(4, 10, requires_grad=True) if fn is sc.distill else z, ids, f(4, 2, dual=True))
        refused("temperature", fn, z, ids, t, temperature=f((), dual=True))
    refused("weights", sc.distill_grad, z, ids, t, f(4, dual=True))
    refused("weight", sc.balance_grad, z, ids, f((), dual=True))
    refused("out", sc.balance_grad, z, ids, out=f(4, 10, dual=True))


@pytest.mark.parametrize("kind,quantize,dequantize,product,widths", [
    (sc.MXRows, sc.mx_quantize, sc.mx_dequantize, sc.mx_product, (128, 8)),
    (sc.ByteRows, sc.byte_quantize, sc.byte_dequantize, sc.byte_product, (256, 4))])
def test_rows_and_products(f, kind, quantize, dequantize, product, widths):
    rows = kind(*(f(6, w, dtype=torch.uint8) for w in widths), 200)
    refused("X", quantize, f(6, 200, dual=True))
    refused("A", product, f(3, 200, dual=True), rows)
    refused("bias", product, f(3, 200), rows, bias=f(6, dual=True))
    refused("out", product, f(3, 200), rows, out=f(3, 6, dual=True))
    refused("out", dequantize, rows, out=f(6, 200, dual=True))
