"""Every way of cutting an MXFP4 product up, without any tolerance.

x and w hold whole numbers times their blocks' scales of 1, 2 or 4 and 1 or 2:
every product is a whole number of at most 36 * 8, and the sums of up to 31512
of them stay below 2^24, so fp32 holds every partial sum exactly, in any order.
A block left out, taken twice, or multiplied with another block's scale shows.
"""
import pytest
import torch

import mx_reference
import mx_rules
import sparse_bf16_delta_amd as sbd

pytestmark = pytest.mark.gpu


def whole(rows, cols, scales, seed):
    """Whole numbers up to 6 times one of `scales` per block, a 6 in each block."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    grid = torch.tensor([0.0, 1, 2, 3, 4, 6], device="cuda")
    x = grid[torch.randint(0, 6, (rows, cols), generator=g, device="cuda")]
    x[torch.rand(rows, cols, generator=g, device="cuda") < 0.5] *= -1
    x[:, ::32] = 6.0
    b = -(-cols // 32)
    s = torch.tensor(scales, device="cuda")[
        torch.randint(0, len(scales), (rows, b), generator=g, device="cuda")]
    return x * s.repeat_interleave(32, dim=1)[:, :cols]


@pytest.mark.parametrize("shape", list(mx_rules.CUTS), ids=str)
def test_sums_are_exact_in_every_cut(shape):
    m, n, k = shape
    assert 36 * 8 * k < 2 ** 24
    x, w = whole(m, k, (1.0, 2.0, 4.0), 1), whole(n, k, (1.0, 2.0), 2)
    qx, qw = sbd.mxfp4_quantize(x), sbd.mxfp4_quantize(w)
    assert torch.equal(sbd.mxfp4_dequantize(qx, torch.float32), x)
    assert torch.equal(sbd.mxfp4_dequantize(qw, torch.float32), w)
    want = x.double() @ w.double().t().contiguous()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        room = torch.full((m * n + 16,), float("nan"), device="cuda", dtype=dtype)
        y = sbd.mxfp4_matmul(qx, qw, out=room[8:-8].view(m, n))
        assert torch.equal(y, want.to(dtype))  # rounded once
        assert bool(room[:8].isnan().all()) and bool(room[-8:].isnan().all())
    # x quantised in the call, from each type (all hold these values)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        assert torch.equal(sbd.mxfp4_matmul(x.to(dtype), qw, out_dtype=torch.float32).double(), want)


def test_the_reference_reads_the_same_values():
    x = whole(70, 333, (1.0, 2.0, 4.0), 3)
    q = sbd.mxfp4_quantize(x)
    b = -(-333 // 32)
    assert torch.equal(mx_reference.values(q.codes.view(70, 16 * b), q.scales.view(70, b), 333),
                       x.double())
