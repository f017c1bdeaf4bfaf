"""What the package's autograd functions share.

Their backward passes run in the library's kernels, so autograd cannot
differentiate them. torch's once_differentiable says so only where the incoming
gradients have a graph of their own: after y.sum(), for one, the result of
torch.autograd.grad(..., create_graph=True) would come back without a graph, and
a penalty on it would be dropped without a word.
"""

from __future__ import annotations

import functools

import torch


class _Once(torch.autograd.Function):
    """Its input, with a graph that raises."""

    @staticmethod
    def forward(ctx, grad, anchor):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("second derivatives are not computed: the function is once_differentiable")


def once_differentiable(backward):
    """For a Function's backward: with create_graph its results raise when they
    are differentiated, whatever the incoming gradients are."""

    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        anchor = torch.zeros((), requires_grad=True)
        return tuple(None if t is None else _Once.apply(t, anchor) for t in out)

    return run
