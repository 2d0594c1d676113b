"""The norms and the linear cross entropy beside autograd: nothing is recorded,
and their calls serve as the two halves of a torch.autograd.Function, whose
gradients are those of the calls by name and of the formulas."""
import pytest
import torch

import optimizer_step_layeradam_amd as la

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        y, stats = la.rms_norm(x, weight)
        ctx.save_for_backward(x, weight, stats)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, stats = ctx.saved_tensors
        return la.rms_norm_backward(dy, x, weight, stats)


class Loss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets):
        loss, dx, dweight = la.linear_cross_entropy_gradients(x, weight, targets)
        ctx.save_for_backward(dx, dweight)
        return loss

    @staticmethod
    def backward(ctx, scale):
        dx, dweight = ctx.saved_tensors
        return scale * dx, scale * dweight, None


def test_nothing_is_recorded():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(20, 64, device="cuda", generator=gen).to(BF).requires_grad_()
    w = torch.randn(300, 64, device="cuda", generator=gen).to(BF).requires_grad_()
    g = torch.ones(64, device="cuda", requires_grad=True)
    y = torch.randint(0, 300, (20,), device="cuda", generator=gen)
    out, stats, s = la.layer_norm(x, g, g, residual=x)
    results = [out, stats, s, *la.layer_norm_backward(out, s, g, stats), *la.rms_norm(x, g),
               la.linear_cross_entropy(x, w, y), *la.linear_cross_entropy_gradients(x, w, y)]
    assert not any(t.requires_grad for t in results)


def test_as_functions_of_autograd():
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(3, 20, 64, device="cuda", generator=gen).to(BF).requires_grad_()
    w = (0.3 * torch.randn(300, 64, device="cuda", generator=gen)).to(BF).requires_grad_()
    g = (1 + 0.2 * torch.randn(64, device="cuda", generator=gen)).to(BF).requires_grad_()
    y = torch.randint(0, 300, (3, 20), device="cuda", generator=gen)
    loss = Loss.apply(RmsNorm.apply(x, g), w, y)
    got = torch.autograd.grad(loss, (x, g, w))
    with torch.no_grad():
        out, stats = la.rms_norm(x, g)
        _, dout, dw = la.linear_cross_entropy_gradients(out, w, y)
        dx, dg = la.rms_norm_backward(dout, x, g, stats)
    for p, q in zip(got, (dx, dg, dw)):
        assert torch.equal(p, q)
    xd, gd, wd = (t.detach().double().requires_grad_() for t in (x, g, w))
    od = xd * (xd.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gd
    want = torch.autograd.grad(torch.nn.functional.cross_entropy(
        od.reshape(60, 64) @ wd.T, y.reshape(60)), (xd, gd, wd))
    # out, g of the softmax and dout are rounded to 16 bits on the way, and the gradient
    # itself, each by half a step (2^-8) at most: by the 2-norm, which the products between
    # do not make grow, 4 halves
    for p, e in zip(got, want):
        assert float((p.double() - e).norm() / e.norm()) < 4 * 2.0 ** -8
