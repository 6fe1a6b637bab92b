"""silu(gate) * up of the MXFP4 product where the gate is far below zero and up
is large, so that the result is an ordinary number.

Gates and ups are sums of a few MXFP4 values that fp32 holds exactly, so only
the activation rounds: its exponential by 2^-21 and, from the rounded product with
log2(e), |gate| 2^-23; the division (2^-22) and the other roundings by 2^-21
together. The result is rounded once; below its type's normal numbers it is off by
half a step of those (2^-134 for bf16, 2^-150 for fp32) and by one of fp32's."""
import pytest
import torch

from sigmoid_bias_top_b200 import mx
from tests import mx_ref as R

pytestmark = pytest.mark.gpu


def check(y, g, u, dtype):
    want = g * torch.sigmoid(g) * u
    eps = torch.finfo(dtype).eps / 2
    rel = (g.abs().clamp_max(256) + 8) * 2.0 ** -23      # no exponential left above
    step = 2.0 ** -134 if dtype is torch.bfloat16 else 2.0 ** -150
    err = want.abs() * rel
    bound = err + eps * (want.abs() + err) + step + 2.0 ** -149
    worst = (y - want).abs() / bound
    assert worst.max() <= 1, (float(worst.max()), float(g.flatten()[worst.argmax()]))


def pieces(v, n=4):
    """v, up to what n numbers of two bits can hold, as those numbers."""
    out, left = [], abs(v)
    for _ in range(n):
        p = 0.0
        if left > 0:
            e = 2.0 ** torch.tensor(left).log2().floor().item()
            p = 1.5 * e if left >= 1.5 * e else e
        out.append(p if v > 0 else -p)
        left -= p
    return out


def make(rows, I, K):
    gates = torch.linspace(-112, 24, I, dtype=torch.float64)
    ups = torch.tensor([1.0, 1.5 * 2.0 ** 60, -2.0 ** 100])
    w = torch.zeros(2 * I, K)
    for i in range(I):
        for b, p in enumerate(pieces(float(gates[i]))):
            w[i, 32 * b] = p
        w[I + i, 5] = ups[i % 3]                    # of block 0, as a column of its own
    a = torch.zeros(rows, K)
    for r in range(rows):
        a[r, 0:128:32] = (0.5, 1.0, 1.5)[r % 3]
        a[r, 5] = 1.0
    return a, w


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,I,K", [(3, 512, 128), (40, 304, 512), (200, 3264, 128), (200, 3264, 512)])
def test_far_gates(rows, I, K, dtype):
    a, w = make(rows, I, K)
    # no block holds numbers far apart, so every one is held exactly
    qa, qw = mx.quantize(a.cuda()), mx.quantize(w.cuda())
    for q, v in ((qa, a), (qw, w)):
        assert torch.equal(torch.from_numpy(R.values(q.codes.cpu().numpy(), q.scales.cpu().numpy())),
                           v.double())
    y = mx.matmul(qa, qw, silu_mul=True, dtype=dtype).double().cpu()
    p = a.double() @ w.double().t()
    g, u = p[:, :I], p[:, I:]
    check(y, g, u, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,I", [(5, 512), (200, 3264)])
def test_gates_of_every_magnitude(rows, I, dtype):
    """Gates of +-2^-125 to 2^119 beside ups that make the results ordinary."""
    e = torch.arange(I) % 245 - 125                       # of the gates
    up = (-e).clamp(-100, 120)
    w = torch.zeros(2 * I, 128)
    w[:I, 0] = torch.where(torch.arange(I) % 2 == 1, -1.0, 1.0)
    w[I:, 0] = 1.5
    q = mx.quantize(w.cuda())
    shift = torch.cat([e, up]).to(torch.int16)
    block = q.scales[:, 0].cpu().to(torch.int16) + shift
    assert block.min() >= 0 and block.max() < 255
    q.scales[:, 0] = block.to(torch.uint8).cuda()
    a = torch.zeros(rows, 128)
    a[:, 0] = 1.0
    qa = mx.quantize(a.cuda())
    g = (w[:I, 0].double() * 2.0 ** e.double()).expand(rows, I)
    u = (w[I:, 0].double() * 2.0 ** up.double()).expand(rows, I)
    check(mx.matmul(qa, q, silu_mul=True, dtype=dtype).double().cpu(), g, u, dtype)
