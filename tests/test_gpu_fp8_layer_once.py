"""examples/fp8_mlp.py: a second derivative is refused, not left out."""
import pytest
import torch

from test_gpu_fp8_layer import example


@pytest.mark.gpu
def test_a_second_derivative_is_refused():
    ex = example()
    torch.manual_seed(5)
    layer = ex.Layer(256, 344)
    x = torch.randn(90, 256, device="cuda").to(torch.bfloat16).requires_grad_()
    loss = layer(x).float().square().sum()
    (g,) = torch.autograd.grad(loss, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (loss + g.float().square().sum()).backward()
