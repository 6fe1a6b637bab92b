"""The balance loss inside a training step: beside another loss under a second
differentiation."""
import pytest
import torch

from sigmoid_bias_top_b200 import balance

pytestmark = pytest.mark.gpu


def make(n=30, E=16, k=3, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(n, E, generator=g, device="cuda").requires_grad_()
    idx = torch.rand(n, E, generator=g, device="cuda").topk(k, 1).indices.int()
    return logits, idx


def test_a_second_derivative_is_refused_beside_other_losses():
    """The other loss has one, so a gradient without a graph would leave the
    balance loss's part out of it without a word."""
    logits, idx = make()
    first = balance.balance_loss(logits, idx).loss
    want, = torch.autograd.grad(first + (logits ** 3).sum(), logits)
    total = (logits ** 3).sum() + balance.balance_loss(logits, idx).loss
    g, = torch.autograd.grad(total, logits, create_graph=True)
    assert torch.equal(g.detach(), want)           # the first derivative is as without
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(g.square().sum(), logits)
    coef = torch.tensor(0.5, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(balance.balance_loss(logits, idx).loss * coef, logits, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(g.sum(), coef)
