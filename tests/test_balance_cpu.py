"""Balance loss without a GPU: refusals of the C ABI and of the binding, the
workspace's size, and the 64-bit reference's gradient against differences."""
import pytest
import torch

from sigmoid_bias_top_b200 import balance
from tests import mx_ref as R


def test_refusals():
    L = balance.lib()

    def fwd(logits=256, dtype=0, ld=16, idx=256, seq=256, n=8, E=16, k=4, B=2, eps=1e-6, ws=256,
            out=256):
        return L.moe_balance_forward(logits, dtype, ld, idx, seq, n, E, k, B, 1.0, eps, ws, out,
                                     out, out, out, None)

    def bwd(logits=256, dtype=0, ld=16, seq=256, n=8, E=16, k=4, B=2, eps=1e-6, out=256):
        return L.moe_balance_backward(logits, dtype, ld, 256, seq, 256, 256, n, E, k, B, eps, out,
                                      None)
    for call in (fwd, bwd):
        assert call(dtype=2) == -1 and call(n=-1) == -1 and call(B=0) == -1
        assert call(eps=-1.0) == -1 and call(eps=float("nan")) == -1
        assert call(seq=None) == -1                      # two sequences need offsets
        assert call(E=0) == -2 and call(E=257) == -2 and call(k=0) == -2 and call(k=9) == -2
        assert call(k=5, E=4) == -2 and call(ld=15) == -1
        assert call(n=1 << 30) == -2 and call(B=1 << 30) == -2
        assert call(logits=None) == -1 and call(out=None) == -1
    assert fwd(idx=None) == -1 and fwd(ws=None) == -1 and fwd(ws=128) == -3
    assert bwd(n=0, logits=None, out=None) == 0


def test_workspace():
    L = balance.lib()
    assert L.moe_balance_workspace(0, 16, 1) >= 256
    assert L.moe_balance_workspace(1 << 20, 256, 4) > L.moe_balance_workspace(8, 256, 4)
    assert L.moe_balance_workspace(-1, 16, 1) == 0


def test_binding_refuses_other_tensors():
    idx = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        balance.balance_loss(torch.zeros(4, 8), idx)     # not on a GPU
    with pytest.raises(TypeError):
        balance.balance_loss(torch.zeros(4, 8).half(), idx)


def test_reference_gradient():
    g = torch.Generator().manual_seed(0)
    l = torch.randn(11, 6, generator=g, dtype=torch.float64)
    idx = torch.randint(-1, 6, (11, 2), generator=g)
    cuts, h = [0, 3, 3, 10], 1e-6
    ref = R.balance(l, idx, cuts, 0.7, 1e-3)
    for t in range(11):
        for e in range(6):
            d = torch.zeros_like(l)
            d[t, e] = h
            num = (R.balance(l + d, idx, cuts, 0.7, 1e-3)["loss"]
                   - R.balance(l - d, idx, cuts, 0.7, 1e-3)["loss"]) / (2 * h)
            assert abs(float(num - ref["grad"][t, e])) < 1e-8


def test_sizes_past_32_bits_are_refused():
    """Counts whose low 32 bits would look like a small one. The tensors have no
    storage: nothing is allocated and nothing launched."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    big = (1 << 32) + 8
    with FakeTensorMode():
        def ints(*shape):
            return torch.empty(*shape, dtype=torch.int32, device="cuda:0")
        with pytest.raises(ValueError, match="2\\^31"):
            balance.balance_loss(torch.empty(big, 1, device="cuda:0"), ints(big, 1))
        with pytest.raises(ValueError, match="2\\^31"):
            balance.balance_loss(torch.empty(8, 4, device="cuda:0"), ints(8, 1), ints(big))
