"""The package's own once_differentiable, on a function that runs on the CPU."""

import pytest
import torch

from bit_block_scaled_bf16_amd.autograd import once_differentiable


class Square(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, also):
        ctx.save_for_backward(x)
        return x * x

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return 2 * ctx.saved_tensors[0] * dy, None


def test_first_derivatives_are_as_without_it():
    x = torch.tensor([1.0, -3.0], requires_grad=True)
    Square.apply(x, None).sum().backward()
    assert torch.equal(x.grad, torch.tensor([2.0, -6.0])) and not x.grad.requires_grad
    g, = torch.autograd.grad(Square.apply(x, None).sum(), x, create_graph=True)
    assert torch.equal(g, torch.tensor([2.0, -6.0]))


@pytest.mark.parametrize("graph_of_its_own", [False, True])
def test_second_derivatives_raise(graph_of_its_own):
    x = torch.tensor([1.0, -3.0], requires_grad=True)
    y = Square.apply(x, None)
    g, = torch.autograd.grad((y * y if graph_of_its_own else y).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (y.sum() + g.square().sum()).backward()
