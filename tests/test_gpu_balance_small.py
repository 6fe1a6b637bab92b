"""Balance loss of tokens whose scores are all tiny: eps 0 or next to it, and
every logit far below zero, where a row's shares are ordinary numbers although
its scores are next to nothing in fp32.

Tolerances as in test_gpu_balance.py, (E + 544) 2^-24 relative to positive sums.
Next to a larger score of its row, one below 2^-126 may be off by as much, that
is 2^-126 of the row's total: 2^-94 for totals of 2^-32 and more, below which
scores are formed in a larger scale."""
import pytest
import torch

from sigmoid_bias_top_b200 import balance
from tests import mx_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(logits, idx, cuts, eps, coef=1.5):
    n, E = logits.shape
    logits = logits.clone().requires_grad_()
    r = balance.balance_loss(logits, idx, torch.tensor(cuts, dtype=torch.int32, device="cuda"),
                             coef=coef, eps=eps)
    grad, = torch.autograd.grad(r.loss, logits)
    l = logits.detach().double().cpu()
    ref = R.balance(l, idx.cpu(), cuts, coef, eps)
    tol, low = (E + 544) * 2.0 ** -24, 2.0 ** -94
    assert torch.equal(r.counts.cpu().double(), ref["counts"])
    torch.testing.assert_close(r.prob.double().cpu(), ref["prob"], rtol=tol, atol=low)
    torch.testing.assert_close(r.loss.detach().double().cpu(), ref["loss"].double(), rtol=tol,
                               atol=low)
    # the gradient is (g - sum g p) p (1 - s): the cancelling difference is off by
    # tol of g + sum g p, and p as above
    s = torch.sigmoid(l)
    p = s / (s.sum(1, keepdim=True) + eps)
    out = torch.finfo(grad.dtype).eps / 2
    live = sum(b > a for a, b in zip(cuts, cuts[1:]))
    for b, (t0, t1) in enumerate(zip(cuts, cuts[1:])):
        g = coef / live * E * ref["counts"][b] / (idx.shape[1] * (t1 - t0) ** 2)
        pb = p[t0:t1]
        amp = g + (g * pb).sum(1, keepdim=True)
        bound = amp * (2 * tol * pb + low) * (1 + out) + out * ref["grad"][t0:t1].abs() + 1e-38
        worst = (grad[t0:t1].double().cpu() - ref["grad"][t0:t1]).abs() / bound
        assert worst.max() <= 1, (b, float(worst.max()))


def selected(n, E, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(n, E, generator=g, device="cuda").topk(k, 1).indices.int()


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -133, 2.0 ** -60])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [1, 4, 16, 40, 256])
def test_rows_of_one_tiny_score(E, dtype, eps):
    """Every expert alike, at both sides of where fp32 scores become subnormal."""
    logits = torch.empty(9, E, device="cuda")
    for t, v in enumerate([-21, -23, -70, -87, -88, -89, -95, -103, 0]):
        logits[t] = v
    check(logits.to(DT[dtype]), selected(9, E, min(E, 3), E), [0, 4, 9], eps)


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -133, 1e-6])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [2, 24, 130])
def test_rows_of_uneven_tiny_scores(E, dtype, eps):
    """Tiny and ordinary rows in one warp, single large scores in tiny rows."""
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = -104 + 20 * torch.rand(61, E, generator=g, device="cuda")
    logits[::5] += 80
    logits[3::7, 0] = -15
    logits[4::7, E - 1] = 2
    logits = logits.to(DT[dtype]).clamp_min(-104)
    check(logits, selected(61, E, 2, E), [0, 1, 33, 61], eps)


def test_a_tiny_row_beside_rows_without_a_score():
    logits = torch.full((6, 8), -95.0, device="cuda")
    logits[1], logits[2, :7], logits[4] = float("-inf"), float("-inf"), -1000.0
    idx = selected(6, 8, 2, 1)
    x = logits.clone().requires_grad_()
    r = balance.balance_loss(x, idx, eps=0.0)
    grad, = torch.autograd.grad(r.loss, x)
    share = torch.full((6, 8), 0.125, dtype=torch.float64)
    share[1], share[2, :7], share[2, 7], share[4] = 0, 0, 1, 0
    tol = 552 * 2.0 ** -24
    torch.testing.assert_close(r.prob[0].double().cpu(), share.mean(0), rtol=tol, atol=0)
    assert torch.isfinite(grad).all() and not grad[1].any() and not grad[4].any()
