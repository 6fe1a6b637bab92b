"""silu(gate) * up of the MXFP4 product where the gate is far below zero and up
is large, so that the result is an ordinary number.

Gates and ups are sums of a few MXFP4 values that fp32 holds exactly, so only
the activation rounds. For bf16 the argument of the exponential, up to 256 as a
power of 2, is off by 2^-16 from the rounded log2(e) and the rounded product, so
the exponential by 2^-16 and, with the division, 2^-21. For fp32 it is 2^-21 and
|gate| 2^-23 for the exponential, 2^-22 for the division and 2^-21 for the other
roundings. silu(gate) is an fp32 number, off by a step of its subnormal ones
(2^-149), times up. The result is rounded once; below its type's normal numbers it
is off by half a step of those (2^-134 for bf16, 2^-150 for fp32) and by one of
fp32's."""
import pytest
import torch

from sigmoid_bias_top_b200 import mx
from tests import mx_ref as R

pytestmark = pytest.mark.gpu


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
    want = g * torch.sigmoid(g) * u
    bf16 = dtype is torch.bfloat16
    eps = torch.finfo(dtype).eps / 2
    rel = 2.0 ** -16 + 2.0 ** -21 if bf16 else (g.abs() + 8) * 2.0 ** -23
    step = 2.0 ** -134 if bf16 else 2.0 ** -150
    err = want.abs() * rel + u.abs() * 2.0 ** -149
    bound = err + eps * (want.abs() + err) + step + 2.0 ** -149
    worst = ((y - want).abs() / bound)
    assert worst.max() <= 1, (float(worst.max()), float(g.flatten()[worst.argmax()]))
