"""The balance loss inside a training step: beside another loss under a second
differentiation, and with its counts summed in place over ranks."""
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


def test_counts_changed_before_the_backward_pass():
    """A collective sums them in place without autograd's knowledge (.data does
    the same here); the gradient is that of this rank's own counts."""
    logits, idx = make(300, 64, 4)
    for off in (None, torch.tensor([0, 100, 100, 290], dtype=torch.int32, device="cuda")):
        r = balance.balance_loss(logits, idx, off)
        want, = torch.autograd.grad(r.loss, logits)
        r = balance.balance_loss(logits, idx, off)
        r.counts.data.mul_(8)
        r.prob.data.zero_()
        got, = torch.autograd.grad(r.loss, logits)
        assert torch.equal(got, want)
        r = balance.balance_loss(logits, idx, off)
        r.counts.add_(1)                           # known to autograd
        assert torch.equal(torch.autograd.grad(r.loss, logits)[0], want)
