"""The balance loss's C entry points without a GPU: arguments that they refuse
before any device work."""
from sigmoid_bias_top_b200 import balance


def forward_kept(n=8, E=16, k=4, B=2, seq=256, out=256, kept=256):
    return balance.lib().moe_balance_forward_kept(256, 0, E, 256, seq, n, E, k, B, 1.0, 1e-6, 256, out,
                                                  out, out, out, kept, None)


def test_forward_kept_refusals():
    assert forward_kept(kept=None) == -1 and forward_kept(out=None) == -1
    assert forward_kept(seq=None) == -1 and forward_kept(n=-1) == -1
    assert forward_kept(E=257) == -2 and forward_kept(k=9) == -2


def test_sizes_whose_sums_would_pass_32_bits():
    """Indices are 32-bit and run past the end by a chunk or a step; the largest
    sizes are refused, those below are not (no output there: -1, after the sizes)."""
    L = balance.lib()
    for top in (1 << 30, (1 << 31) - 1024, (1 << 31) - 1):
        for n, B in ((top, 1), (8, top)):
            assert forward_kept(n=n, B=B, E=1, k=1) == -2
            assert L.moe_balance_forward(256, 0, 1, 256, 256, n, 1, 1, B, 1.0, 0.0, 256, 256, 256, 256,
                                         256, None) == -2
            assert L.moe_balance_backward(256, 0, 1, 256, 256, 256, 256, n, 1, 1, B, 0.0, 256,
                                          None) == -2
            assert L.moe_balance_workspace(n, 1, B) == 0
    top = (1 << 30) - 1
    for n, B in ((top, 1), (8, top)):
        assert forward_kept(n=n, B=B, E=1, k=1, out=None) == -1
        assert L.moe_balance_backward(256, 0, 1, 256, 256, 256, 256, n, 1, 1, B, 0.0, None, None) == -1
        assert L.moe_balance_workspace(n, 1, B) > 8 * B
