"""The balance loss's autograd node without a GPU: the C entry points are stood in
for by ones that launch nothing, so values mean nothing here and the graph does."""
import pytest
import torch

from sigmoid_bias_top_b200 import balance


class Entries:
    def moe_balance_workspace(self, n, E, B):
        return 1024

    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def no_device(monkeypatch):
    monkeypatch.setattr(balance, "lib", Entries)
    monkeypatch.setattr(balance, "_raw_stream", lambda index: 0)


def apply(logits):
    return balance._BalanceLoss.apply(logits, torch.zeros(logits.shape[0], 2, dtype=torch.int32), None,
                                      1.0, 1e-6)[0]


def test_a_second_derivative_is_refused(no_device):
    logits = torch.randn(5, 4).requires_grad_()
    total = (logits ** 3).sum() + apply(logits)
    g, = torch.autograd.grad(total, logits, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(g.sum(), logits)
    coef = torch.tensor(0.5, requires_grad=True)
    g, = torch.autograd.grad(apply(logits) * coef, logits, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(g.sum(), coef)


def test_a_first_derivative_has_no_graph(no_device):
    logits = torch.randn(5, 4).requires_grad_()
    g, = torch.autograd.grad(apply(logits * 2.0), logits)
    assert not g.requires_grad
    with torch.no_grad():
        assert not apply(logits).requires_grad
