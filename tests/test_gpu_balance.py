"""Balance loss, per-expert counts and the gradient of the logits on the GPU
against the 64-bit reference (tests/mx_ref.py).

Tolerances, relative to positive sums: a score carries a few roundings, a row's
sum of scores at most E more, a chunk's sum of shares at most its tokens over
the rows that a warp holds (under 512), each 2^-24: TOL = (E + 512 + 32) 2^-24.
The gradient's (g - sum g p) may cancel, so its error is counted against
(g + sum g p) times the same factors, plus the rounding of the stored type."""
import pytest
import torch

from sigmoid_bias_top_b200 import MoeLayer, balance, route_noalloc, workloads as W
from tests import mx_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(n, E, k, dtype, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (spread * torch.randn(n, E, generator=g, device="cuda")).to(DT[dtype])
    idx = torch.rand(n, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    return logits, idx.contiguous()


def offs(*cuts):
    return torch.tensor(cuts, dtype=torch.int32, device="cuda")


def check(r, grad, logits, idx, offsets, coef, eps, scale=1.0):
    E = logits.shape[1]
    ref = R.balance(logits.detach().double().cpu(), idx.cpu(), offsets, coef, eps)
    tol = (E + 512 + 32) * 2.0 ** -24
    assert torch.equal(r.counts.cpu().double(), ref["counts"])
    torch.testing.assert_close(r.prob.double().cpu(), ref["prob"], rtol=tol, atol=1e-38)
    torch.testing.assert_close(r.loss.detach().double().cpu(), ref["loss"].double(), rtol=tol,
                               atol=1e-38)
    # |error of grad| <= tol * (g + sum g p) / total * slope, and its own rounding
    n = logits.shape[0]
    l = logits.detach().double().cpu()
    s = torch.sigmoid(l)
    total = s.sum(1, keepdim=True) + eps
    total = torch.where(total > 0, total, float("inf"))   # no share, no gradient, no error
    live = sum(offsets[b + 1] > offsets[b] for b in range(len(offsets) - 1))
    amp = torch.zeros(n, E, dtype=torch.float64)
    for b in range(len(offsets) - 1):
        t0, t1 = offsets[b], offsets[b + 1]
        if t1 > t0:
            g = coef / live * E * ref["counts"][b] / (idx.shape[1] * (t1 - t0) ** 2)
            p = s[t0:t1] / total[t0:t1]
            amp[t0:t1] = ((g + (g * p).sum(1, keepdim=True)) / total[t0:t1]
                          * s[t0:t1] * torch.sigmoid(-l[t0:t1]))
    eps_out = 2.0 ** -8 if grad.dtype == torch.bfloat16 else 2.0 ** -24
    want = ref["grad"] * scale
    bound = abs(scale) * (tol * amp * (1 + eps_out)) + eps_out * want.abs() + 1e-38
    worst = (grad.double().cpu() - want).abs() / bound
    assert not worst.numel() or worst.max() <= 1, float(worst.max())


CASES = [
    (1, 8, 1, (0, 1)), (1, 1, 1, (0, 1)), (5, 16, 4, (0, 5)), (64, 16, 4, (0, 1, 1, 40, 63, 64)),
    (100, 40, 3, (0, 100)), (333, 64, 4, (0, 7, 200, 200, 333)), (17, 256, 8, tuple(range(18))),
    (2000, 12, 2, (0, 1999, 2000)), (513, 129, 5, (0, 512, 513)), (9000, 64, 4, (0, 8, 16, 9000)),
    (40, 64, 8, (5, 11, 30)),              # tokens before the first and behind the last sequence
    (30, 24, 2, (0, 0, 0)), (12, 24, 2, (12, 12, 12)),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,E,k,cuts", CASES)
def test_against_reference(n, E, k, cuts, dtype):
    logits, idx = make(n, E, k, dtype, n + E, 2.0)
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx, offs(*cuts), coef=0.3, eps=1e-6)
    grad, = torch.autograd.grad(r.loss, logits)
    assert grad.dtype == logits.dtype and grad.shape == logits.shape
    check(r, grad, logits, idx, list(cuts), 0.3, 1e-6)
    again = balance.balance_loss(logits, idx, offs(*cuts), coef=0.3, eps=1e-6)
    assert torch.equal(again.loss, r.loss) and torch.equal(again.prob, r.prob)
    assert torch.equal(torch.autograd.grad(again.loss, logits)[0], grad)


def test_no_offsets_is_one_sequence():
    logits, idx = make(77, 32, 4, "f32")
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx)
    grad, = torch.autograd.grad(r.loss * 3.0, logits)
    check(r, grad, logits, idx, [0, 77], 1.0, 1e-6, scale=3.0)


def test_empty_batch():
    logits, idx = make(0, 16, 2, "f32")
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx)
    assert r.loss.item() == 0 and not r.counts.any() and not r.prob.any()
    assert torch.autograd.grad(r.loss, logits)[0].shape == (0, 16)


def test_dropped_slots_are_not_counted():
    logits, idx = make(50, 16, 4, "f32")
    idx[3] = -1
    idx[7, 2] = 16
    idx[8, 0] = 2 ** 31 - 1
    idx[9, 1] = -2 ** 31
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx, offs(0, 20, 50))
    assert r.counts.sum().item() == 200 - 7
    check(r, torch.autograd.grad(r.loss, logits)[0], logits, idx, [0, 20, 50], 1.0, 1e-6)


def test_extreme_logits():
    """Scores of 0 and 1, a row whose scores all underflow with eps 0 (no share
    and no gradient), logits of the type's lowest value and -inf."""
    logits, idx = make(12, 16, 2, "f32", 3, 30.0)
    logits[2] = -200.0
    logits[3] = float("-inf")
    logits[4, :8] = torch.finfo(torch.float32).min
    logits[5] = torch.finfo(torch.float32).max
    logits.requires_grad_()
    for eps in (0.0, 1e-6):
        r = balance.balance_loss(logits, idx, offs(0, 6, 12), eps=eps)
        grad, = torch.autograd.grad(r.loss, logits)
        assert torch.isfinite(grad).all() and torch.isfinite(r.loss)
        # expf underflows to 0 below -104: the reference gets the same scores
        ref_logits = torch.where(logits.detach() < -104, float("-inf"), logits.detach().double())
        check(r, grad, ref_logits, idx, [0, 6, 12], 1.0, eps)


def test_tokens_of_no_sequence_may_hold_anything():
    """NaN, infinities and the types' lowest values before the first sequence and
    behind the last reach neither the loss nor a gradient."""
    for dtype in ("f32", "bf16"):
        for E in (16, 37, 256):
            logits, idx = make(70, E, 4, dtype, E)
            logits[:7], logits[60:] = float("nan"), float("inf")
            logits[65:] = torch.finfo(DT[dtype]).min
            idx[:7] = -1
            logits.requires_grad_()
            r = balance.balance_loss(logits, idx, offs(7, 30, 30, 60), coef=2.0)
            grad, = torch.autograd.grad(r.loss, logits)
            assert torch.isfinite(r.loss) and torch.isfinite(r.prob).all()
            assert not grad[:7].any() and not grad[60:].any()
            check(r, grad[7:60], logits[7:60], idx[7:60], [0, 23, 23, 53], 2.0, 1e-6)


def test_a_bad_token_stays_in_its_sequence():
    logits, idx = make(50, 32, 4, "f32")
    logits[12, 3] = float("nan")
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx, offs(0, 20, 50))
    grad, = torch.autograd.grad(r.loss, logits)
    assert torch.isnan(r.loss) and torch.isnan(r.prob[0]).all()
    assert torch.isfinite(r.prob[1]).all() and torch.isnan(grad[12]).all()
    rest = [t for t in range(50) if t != 12]
    assert torch.isfinite(grad[rest]).all()


def test_loss_is_an_ordinary_tensor():
    """Added to in place, detached, without a gradient wanted; a second backward
    of the backward is refused."""
    logits, idx = make(20, 16, 2, "f32")
    plain = balance.balance_loss(logits, idx)
    assert not plain.loss.requires_grad
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx, coef=0.5)
    loss = r.loss
    loss += (logits * logits).sum()
    loss.backward()
    alone, = torch.autograd.grad(balance.balance_loss(logits, idx, coef=0.5).loss, logits)
    torch.testing.assert_close(logits.grad, alone + 2 * logits.detach(), rtol=1e-5, atol=1e-6)
    assert not r.counts.requires_grad and not r.prob.requires_grad
    g, = torch.autograd.grad(balance.balance_loss(logits, idx).loss, logits, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), logits)
    with torch.no_grad():
        assert torch.equal(balance.balance_loss(logits, idx).loss, plain.loss)


def test_two_streams_at_once():
    cases = [make(3000, 64, 4, "f32", i) for i in (1, 2)]
    want = []
    for logits, idx in cases:
        logits.requires_grad_()
        r = balance.balance_loss(logits, idx, offs(0, 1000, 3000))
        want.append((r.loss.detach().clone(), torch.autograd.grad(r.loss, logits)[0].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    o = offs(0, 1000, 3000)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (logits, idx) in zip(streams, cases):
            with torch.cuda.stream(s):
                r = balance.balance_loss(logits, idx, o)
                got.append((r.loss.detach(), torch.autograd.grad(r.loss, logits)[0]))
    torch.cuda.synchronize()
    for i, (loss, grad) in enumerate(got):
        assert torch.equal(loss, want[i % 2][0]) and torch.equal(grad, want[i % 2][1])


def test_many_sequences():
    """More sequences than chunks, most of one token, some empty."""
    n = 5000
    logits, idx = make(n, 24, 3, "f32", 8)
    cuts = torch.cat([torch.arange(0, 4000), torch.arange(4000, n, 7), torch.tensor([n, n, n])])
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx, cuts.int().cuda())
    check(r, torch.autograd.grad(r.loss, logits)[0], logits, idx, cuts.tolist(), 1.0, 1e-6)


def test_long_batch():
    """More tokens than the GPU has chunks for at their usual size."""
    n = 650_000
    logits, idx = make(n, 8, 2, "bf16", 4)
    logits.requires_grad_()
    cuts = (0, 3, n - 70_001, n)
    r = balance.balance_loss(logits, idx, offs(*cuts))
    check(r, torch.autograd.grad(r.loss, logits)[0], logits, idx, list(cuts), 1.0, 1e-6)


def test_strided_and_unaligned_logits():
    base = torch.randn(60, 100, device="cuda")
    for view in (base[:, :64], base[::2, 4:68], base[:, 1:65], base[:, 3:40], base.t()[:, :24],
                 base[:1, :16].expand(30, 16)):
        n, E = view.shape
        _, idx = make(n, E, 4, "f32")
        leaf = view.detach().requires_grad_()
        r = balance.balance_loss(leaf, idx, offs(0, n // 3, n))
        grad, = torch.autograd.grad(r.loss, leaf)
        check(r, grad, view, idx, [0, n // 3, n], 1.0, 1e-6)


def test_gradient_against_differences():
    """Central differences of the 64-bit loss (the counts held fixed)."""
    logits, idx = make(9, 12, 3, "f32", 5)
    logits.requires_grad_()
    r = balance.balance_loss(logits, idx, offs(0, 4, 9), coef=2.0)
    grad, = torch.autograd.grad(r.loss, logits)
    l, i, h = logits.detach().double().cpu(), idx.cpu(), 1e-5
    scale = float(grad.abs().max())
    for t, e in [(0, 0), (3, 11), (4, 5), (8, 2), (6, 7)]:
        d = torch.zeros_like(l)
        d[t, e] = h
        num = (R.balance(l + d, i, [0, 4, 9], 2.0, 1e-6)["loss"]
               - R.balance(l - d, i, [0, 4, 9], 2.0, 1e-6)["loss"]) / (2 * h)
        # differences: h^2 of the third derivative and 1e-16 / h of the loss
        assert abs(float(num) - float(grad[t, e])) <= 1e-4 * scale


def test_training_step_and_refusals():
    """A router's gradient through its matrix, as a training step takes it."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(64, 32, generator=g, device="cuda")
    w = torch.randn(16, 32, generator=g, device="cuda").requires_grad_()
    logits = x @ w.t()
    idx = torch.sigmoid(logits.detach()).topk(4, 1).indices.int()
    r = balance.balance_loss(logits, idx, offs(0, 30, 64), coef=0.1)
    r.loss.backward()
    ref = R.balance(logits.detach().double().cpu(), idx.cpu(), [0, 30, 64], 0.1, 1e-6)
    want = ref["grad"].t() @ x.double().cpu()
    torch.testing.assert_close(w.grad.double().cpu(), want, rtol=1e-3,
                               atol=1e-5 * float(want.abs().max()))
    with pytest.raises(ValueError):
        balance.balance_loss(logits, idx.long())
    with pytest.raises(ValueError):
        balance.balance_loss(logits, idx[:5])
    with pytest.raises(TypeError):
        balance.balance_loss(logits.half(), idx)
    with pytest.raises(ValueError):
        balance.balance_loss(logits, idx, offs(0, 64).long())
    with pytest.raises(Exception):
        balance.balance_loss(torch.zeros(4, 300, device="cuda"), idx[:4])


def test_counts_of_the_routers_selection():
    """The counts of a routed batch are those by which the layer's dispatch
    groups its rows."""
    w = W.DECODE.scaled(n_tokens=100)
    layer = W.make_layer(w, 0, "cuda")
    x = W.make_x(w, "cuda")
    idx, _ = route_noalloc(x, layer, w.top_k, w.eps)
    m = MoeLayer(layer, w.top_k, w.eps, max_tokens=100)
    m(x)
    offsets = m.debug_routing(100)["offsets"]
    logits = torch.randn(100, w.n_experts, device="cuda")
    r = balance.balance_loss(logits, idx)
    assert torch.equal(r.counts[0].cumsum(0).int(), offsets[1:])
    m.close()


def test_captured_step():
    """Forward and backward captured together; replays read new contents. The
    eager graph of the same leaf is gone before the capture."""
    logits, idx = make(300, 64, 4, "f32")
    logits.requires_grad_()
    o = offs(0, 100, 300)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                     # warm-up, as captures want it
        torch.autograd.grad(balance.balance_loss(logits, idx, o).loss, logits)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = balance.balance_loss(logits, idx, o)
        grad, = torch.autograd.grad(r.loss, logits)
    for seed in (1, 2):
        l, i = make(300, 64, 4, "f32", seed)
        with torch.no_grad():
            logits.copy_(l)
        idx.copy_(i)
        o.copy_(offs(0, 100 + 50 * seed, 300))
        g.replay()
        torch.cuda.synchronize()
        check(r, grad, logits, idx, [0, 100 + 50 * seed, 300], 1.0, 1e-6)
