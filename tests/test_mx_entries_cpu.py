"""The MXFP4 entry points without a GPU: widths past what the product takes."""
import ctypes

import sigmoid_bias_top_b200 as sb
from sigmoid_bias_top_b200 import mx


def test_product_width():
    """A row's steps along K are counted in 32 bits, and a tile is one bounded
    wait of the roles that do not step along it. The largest width passes the
    shapes' check (no output there: -1, after it)."""
    def call(K, out):
        return mx.lib().moe_mx_matmul(256, 256, 256, 256, 256, 4, K, 2, 64, 0, out, 1, None)
    for K in (1 << 22, 128):
        assert call(K, None) == -1
    for K in ((1 << 22) + 128, 1 << 24, (1 << 31) - 384, (1 << 31) - 128):
        assert call(K, 256) == -2 and call(K, None) == -2


def test_layer_width():
    L = sb.lib()

    def create(I, dtype=sb.MOE_MXFP4):
        h = ctypes.c_void_p(7)
        # no scales: -1, after the shapes
        w = sb.MoeWeights(dtype, 256, 256, 256, 256, 256, 1.0, None, None)
        return L.moe_create(128, 1, I, 1, 1e-6, ctypes.byref(w), 16, ctypes.byref(h))
    assert create(1 << 22) == -1
    assert create((1 << 22) + 128) == -2 and create(1 << 28) == -2
    assert create((1 << 22) + 128, sb.MOE_FP8_BLOCK) == -1     # other layers as they were


def test_selftest_timeout_refusals():
    def call(timeout_us=1000, withheld=1, rows=4, K=256, out=256):
        return mx.lib().moe_mx_selftest_timeout(256, 256, 256, 256, 256, rows, K, 2, 64, 0, out, 1,
                                                timeout_us, withheld, None)
    assert call(timeout_us=0) == -1 and call(timeout_us=1000001) == -1
    assert call(withheld=-1) == -1 and call(withheld=11) == -1
    assert call(out=None) == -1 and call(K=64) == -2
