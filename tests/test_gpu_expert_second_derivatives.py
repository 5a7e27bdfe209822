"""The example's routing has a first derivative only: a second one is refused, not taken for zero."""
import pytest

pytestmark = pytest.mark.gpu


def test_second_derivatives_are_refused():
    import torch
    from examples.expert_training_step import Experts
    layer = Experts(100, 16, 16, 8, 2)
    x = torch.randn(100, 16, device="cuda")
    first = torch.autograd.grad(layer(x).square().mean(), (layer.router, layer.up), create_graph=True)
    total = sum(g.square().sum() for g in first)
    # the router's gradient depends on `up` through the gradient of the routing's weights
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(total, layer.up, retain_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        total.backward()
