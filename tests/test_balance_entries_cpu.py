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
