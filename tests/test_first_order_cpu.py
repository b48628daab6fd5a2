"""Backward passes whose results are kernels' outputs: a second derivative raises, first ones are as they were."""
import pytest
import torch

from mxfp8_precision_moe_gb300 import _first_order


class Double(torch.autograd.Function):

    @staticmethod
    def forward(ctx, a, b):
        ctx.save_for_backward(a, b)
        return a * b

    @staticmethod
    @_first_order
    def backward(ctx, g):
        a, b = ctx.saved_tensors
        return g * b if ctx.needs_input_grad[0] else None, g * a if ctx.needs_input_grad[1] else None


def leaves():
    return torch.tensor([2.0, 3.0], requires_grad=True), torch.tensor([5.0, 7.0], requires_grad=True)


def test_first_derivatives():
    a, b = leaves()
    Double.apply(a, b).sum().backward()
    assert a.grad.tolist() == [5, 7] and b.grad.tolist() == [2, 3] and not a.grad.requires_grad
    ga, = torch.autograd.grad(Double.apply(a, b.detach()).sum(), a, create_graph=True)
    assert ga.tolist() == [5, 7]


@pytest.mark.parametrize("constant", [True, False])
def test_second_derivatives_raise(constant):
    """Whether the incoming gradient is a constant (a sum's) or depends on the leaves (a square's)."""
    a, b = leaves()
    out = Double.apply(a, b)
    ga, = torch.autograd.grad(out.sum() if constant else out.square().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (ga.sum() + b.sum()).backward()  # without the error b's gradient would be 1


def test_create_graph_without_a_second_derivative():
    a, b = leaves()
    Double.apply(a, b).sum().backward(create_graph=True)
    assert a.grad.tolist() == [5, 7] and b.grad.tolist() == [2, 3]
