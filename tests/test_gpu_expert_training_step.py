"""The example's training step with experts: its gradients against torch's own autograd of the same layer, and
that it learns with its gradients clipped."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def test_gradients_match_autograd():
    import torch
    from examples.expert_training_step import Experts
    torch.manual_seed(3)
    torch.backends.cuda.matmul.allow_tf32 = False
    t, e, k = 300, 16, 2
    layer = Experts(t, 32, 48, e, k)
    layer.bias.copy_(0.05 * torch.randn(e, device="cuda"))
    x = torch.randn(t, 32, device="cuda")
    goal = torch.randn(t, 32, device="cuda")
    (layer(x) - goal).square().mean().backward()
    got = [p.grad.clone() for p in layer.parameters()]

    # the same in 64 bits, with the choice that was made and differentiable scores
    ids = layer.route.ids.long()
    w = [p.detach().double().requires_grad_() for p in layer.parameters()]
    xd = x.double()
    s = torch.sigmoid(xd @ w[0]).gather(1, ids)
    s = s / s.sum(-1, keepdim=True)
    out = sum((torch.relu(torch.einsum("td,tdh->th", xd, w[1][ids[:, j]])).unsqueeze(1) @ w[2][ids[:, j]]).squeeze(1)
              * s[:, j:j + 1] for j in range(k))
    (out - goal.double()).square().mean().backward()
    for a, b in zip(got, w):
        # sums of up to 300 x 48 products in 32 bits: 2^-24 times a path of some 500 roundings, against the largest
        assert (a.double() - b.grad).abs().max() <= 500 * 2.0 ** -24 * b.grad.abs().max()


def test_it_learns():
    from examples.expert_training_step import train
    losses, norms = train(steps=60)
    assert np.mean(losses[-10:]) < 0.9 * np.mean(losses[:10])
    assert any(a > 0.05 for a, _ in norms)
    for before, after in norms:
        # clipped to max_norm / (norm + eps) of itself, each element rounded once: a relative 1e-5 at most
        assert after <= min(before, 0.05) * (1 + 1e-5)
