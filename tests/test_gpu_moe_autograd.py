"""The sort's rows and their gradients in a torch.autograd.Function of a user's own, as the package's docstring says:
no call records a graph itself, and with the gradient calls in backward() the gradients are the formulas'."""
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu

H = torch.finfo(torch.bfloat16).eps / 2


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos):
        ctx.save_for_backward(pos)
        xs = x.new_zeros((pos.numel(), x.shape[1]))
        return dg.dg_moe_gather(x, pos, xs=xs)

    @staticmethod
    def backward(ctx, dxs):
        return dg.dg_moe_combine(dxs.contiguous(), *ctx.saved_tensors), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, pos, w):
        ctx.save_for_backward(z, pos, w)
        return dg.dg_moe_combine(z, pos, w)

    @staticmethod
    def backward(ctx, dy):
        dz, dw = dg.dg_moe_combine_grad(dy.contiguous(), *ctx.saved_tensors)
        return dz, None, dw


@pytest.mark.parametrize("M,topk,E,K", [(1, 1, 2, 8), (7, 3, 9, 40), (300, 8, 64, 1032)])
def test_gradients_through_there_and_back(cuda_device, M, topk, E, K):
    g = torch.Generator("cuda").manual_seed(M + K)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16).requires_grad_()
    w = torch.rand((M, topk), generator=g, device="cuda").requires_grad_()
    dy = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand((M, E), generator=g, device="cuda").topk(topk, -1).indices.int()
    ids[torch.rand((M, topk), generator=g, device="cuda") < 0.2] = -1
    _, pos, _ = dg.dg_moe_sort(ids, E)
    assert not dg.dg_moe_gather(x, pos).requires_grad and not dg.dg_moe_combine(x, pos[:, :1].clone(), None).requires_grad
    y = Combine.apply(Gather.apply(x, pos), pos, w)
    y.backward(dy)
    live = (ids >= 0).double()
    xd, wd, dyd = x.detach().double(), w.detach().double() * live, dy.double()
    ref = xd * wd.sum(1, keepdim=True)
    mag = xd.abs() * wd.sum(1, keepdim=True)
    # topk rounded steps in binary32, one rounding to bf16
    assert ((y.detach().double() - ref).abs() <= H * ref.abs() + (topk + 1) * 2.0 ** -24 * 2 * mag).all()
    # each row of dz is rounded to bf16, and their sum
    refx, magx = dyd * wd.sum(1, keepdim=True), dyd.abs() * wd.sum(1, keepdim=True)
    assert ((x.grad.double() - refx).abs() <= H * refx.abs() + (H * (1 + H) + (topk + 1) * 2.0 ** -23) * magx).all()
    refw, magw = (dyd * xd).sum(1, keepdim=True) * live, (dyd * xd).abs().sum(1, keepdim=True) * live
    assert ((w.grad.double() - refw).abs() <= K * 2.0 ** -24 * magw).all()
