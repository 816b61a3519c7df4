"""A clip plan and the gradients of a training loop: those that stay in their
tensors are clipped every step, those that a step made anew are refused."""
import math

import pytest
import torch

import sparse_bf16_delta_amd as sbd

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24


def model():
    torch.manual_seed(0)
    m = torch.nn.Sequential(torch.nn.Linear(37, 64), torch.nn.Linear(64, 5)).cuda()
    return m, torch.optim.SGD(m.parameters(), lr=0.1)


def backward(m, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m(torch.randn(9, 37, generator=g, device="cuda")).square().sum().backward()
    return [p.grad for p in m.parameters()]


def test_gradients_that_stay():
    m, opt = model()
    plan = None
    for step in range(3):
        opt.zero_grad(set_to_none=False)
        grads = backward(m, step)
        plan = plan or sbd.ClipPlan(grads)
        before = [g.double() for g in grads]
        size = math.sqrt(sum(float(b.square().sum()) for b in before))
        assert abs(float(plan.norm(grads)) - size) <= 8 * STEP * size
        assert abs(float(plan.total(grads)) - size ** 2) <= 16 * STEP * size ** 2
        norm = float(plan.run(0.5 * size, grads=grads))
        assert abs(norm - size) <= 8 * STEP * size
        factor = 0.5 * size / (size + 1e-6)
        for g, b in zip(grads, before):
            assert bool(((g.double() - b * factor).abs() <= 12 * STEP * b.abs() + 2.0 ** -149).all())
        opt.step()


def test_gradients_made_anew_are_refused():
    m, opt = model()
    grads = backward(m, 0)
    plan = sbd.ClipPlan(grads)
    opt.zero_grad()  # drops them; the plan keeps the old tensors alive
    new = backward(m, 1)
    assert all(a.data_ptr() != b.data_ptr() for a, b in zip(grads, new))
    before = [g.clone() for g in grads + new]
    for call in (lambda g: plan.run(1e-3, grads=g), plan.norm, plan.total):
        with pytest.raises(ValueError, match="made for"):
            call(new)
        with pytest.raises(ValueError, match="made for"):
            call(new[:1] + grads[1:])
        with pytest.raises(ValueError, match="made for"):
            call(grads[:-1])
        with pytest.raises(ValueError, match="made for"):
            call([None] + grads[1:])
        with pytest.raises(ValueError, match="made for"):
            call([grads[0].t()] + grads[1:])  # the same memory, read otherwise
        with pytest.raises(ValueError, match="made for"):
            call([grads[0].view(torch.int32)] + grads[1:])
    torch.cuda.synchronize()
    for g, b in zip(grads + new, before):
        assert torch.equal(g, b)
    views = [g.view(-1) for g in grads]  # other objects over the same values
    assert float(plan.run(math.inf, grads=views)) == float(sbd.grad_norm(grads))
