"""The linear layer in autograd graphs."""

import pytest

from tests._helpers import announce, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [1, 2])
def test_linear_second_derivative_is_refused(power):
    """The layer's backward pass is not differentiable: a gradient penalty raises
    instead of being dropped."""
    torch = require_gpu()
    from bit_block_scaled_bf16_amd.linear import NVFP4Linear

    announce(f"second derivative of the layer, power {power}")
    layer = NVFP4Linear(64, 32, device="cuda")
    x = torch.randn(32, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    g, = torch.autograd.grad(layer(x).float().pow(power).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (layer.weight.float().sum() + g.float().square().sum()).backward()
