"""The MXFP4 product has no gradient: where one would be lost, the call is
refused instead of returning a result without a graph."""
import pytest
import torch

import sparse_bf16_delta_amd as sbd


def refused(x, w, **out):
    with pytest.raises(ValueError, match="requires a gradient"):
        sbd.mxfp4_matmul(x, w, **out)


def test_refused_before_anything_else():
    w = sbd.mxfp4_empty((4, 64), "cpu")
    x = torch.zeros(2, 64, requires_grad=True)
    refused(x, w)
    refused(x * 2, w)
    refused(torch.zeros(2, 64), w, out=torch.zeros(2, 4, requires_grad=True))
    for call in (lambda: sbd.mxfp4_matmul(x.detach(), w), lambda: sbd.mxfp4_matmul(x.data, w)):
        with pytest.raises(ValueError, match="on a GPU"):  # the next check
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="on a GPU"):
        sbd.mxfp4_matmul(x, w)


@pytest.mark.gpu
def test_the_product_without_recording():
    w = sbd.mxfp4_quantize(torch.randn(40, 64, device="cuda"))
    x = torch.randn(3, 64, device="cuda", requires_grad=True)
    refused(x, w)
    want = sbd.mxfp4_matmul(x.detach(), w)
    with torch.no_grad():
        assert torch.equal(sbd.mxfp4_matmul(x, w), want)
    with torch.inference_mode():
        assert torch.equal(sbd.mxfp4_matmul(x, w), want)
    # a parameter's replica carries no graph, so making one is no loss
    p = torch.nn.Parameter(torch.randn(40, 64, device="cuda"))
    assert torch.equal(sbd.mxfp4_matmul(x.detach(), sbd.mxfp4_quantize(p)),
                       sbd.mxfp4_matmul(x.detach(), sbd.mxfp4_quantize(p.detach())))
