"""MXFP4 operators without a GPU: the C ABI refuses bad arguments before any
device work, the binding refuses tensors it does not take, and the 64-bit
reference that the GPU tests compare with has the format's properties."""
import numpy as np
import pytest
import torch

from sigmoid_bias_top_b200 import mx
from tests import mx_ref as R


def test_quantize_refusals():
    L = mx.lib()

    def call(x=256, dtype=1, rows=4, K=64, ld=64, codes=256, scales=256):
        return L.moe_mx_quantize(x, dtype, rows, K, ld, codes, scales, None)
    assert call(dtype=2) == -1 and call(rows=-1) == -1 and call(x=None) == -1
    assert call(codes=None) == -1 and call(scales=None) == -1
    assert call(K=48) == -2 and call(K=0) == -2 and call(K=-32) == -2
    assert call(rows=1 << 60) == -2
    assert call(ld=32) == -1                        # rows would overlap
    assert call(ld=65) == -3                        # bf16 rows off 16 bytes
    assert call(dtype=0, ld=66) == -3
    assert call(x=264) == -3 and call(codes=264) == -3
    assert call(rows=0, x=None, codes=None, scales=None) == 0


def test_dequantize_refusals():
    L = mx.lib()

    def call(codes=256, scales=256, rows=4, K=64, y=256, dtype=1):
        return L.moe_mx_dequantize(codes, scales, rows, K, y, dtype, None)
    assert call(dtype=2) == -1 and call(rows=-1) == -1 and call(y=None) == -1
    assert call(K=33) == -2
    assert call(y=260) == -3 and call(codes=8) == -3
    assert call(rows=0) == 0


def test_matmul_refusals():
    L = mx.lib()

    def call(a=256, a_s=256, w=256, w_s=256, offs=256, rows=4, K=256, E=2, N=64, silu=0, out=256,
             dtype=1):
        return L.moe_mx_matmul(a, a_s, w, w_s, offs, rows, K, E, N, silu, out, dtype, None)
    assert call(dtype=2) == -1 and call(rows=-1) == -1 and call(silu=2) == -1
    assert call(offs=None) == -1                    # two experts need offsets
    for name in ("a", "a_s", "w", "w_s", "out"):
        assert call(**{name: None}) == -1, name
    assert call(K=64) == -2 and call(K=0) == -2 and call(N=0) == -2 and call(N=24) == -2
    assert call(N=48, silu=1) == -2 and call(E=0) == -2 and call(E=257) == -2
    assert call(rows=1 << 30) == -2 and call(E=256, N=1 << 22) == -2
    assert call(a=264) == -3 and call(w=264) == -3 and call(out=264) == -3
    assert call(a_s=258) == -3 and call(w_s=258) == -3 and call(offs=258) == -3
    assert call(rows=0, a=None, out=None) == 0


def test_binding_refuses_other_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        mx.quantize(x)                               # not on a GPU
    with pytest.raises(TypeError):
        mx.quantize(x.half())
    q = mx.MxTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        mx.dequantize(q)
    with pytest.raises(TypeError):
        mx.matmul(q, q)
    with pytest.raises(TypeError):
        mx.dequantize(q, torch.float16)
    assert q.shape == (4, 64)


def test_reference_rounding():
    """Ties go to the even code, values above 6 saturate, the exponent follows
    the block's largest value."""
    x = np.zeros((1, 32))
    x[0, :16] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.76, -5.01, 7.9, 0.26, 0, 6, 1]
    codes, scales = R.quantize(x)
    assert scales[0, 0] == 127
    v = R.values(codes, scales)[0, :16]
    assert v.tolist() == [4, 0, 1, 1, 2, 2, 4, 4, -0.0, -1, -6, 6, 0.5, 0, 6, 1]
    y = np.full((1, 32), np.nan)
    assert R.quantize(y)[1][0, 0] == 255
    assert R.quantize(np.full((1, 32), 2.0 ** -149))[1][0, 0] == 0
    z, s = R.quantize(np.zeros((1, 32)))
    assert s[0, 0] == 0 and not z.any()


def test_mxfp4_layer_refusals():
    """moe_create checks an MXFP4 layer's shapes, scale arrays and alignment
    before any device work; expert-parallel contexts do not take one."""
    import ctypes

    import sigmoid_bias_top_b200 as sb
    L = sb.lib()

    def create(d=2048, I=1536, scales=(256, 256)):
        h = ctypes.c_void_p(7)
        w = sb.MoeWeights(sb.MOE_MXFP4, 256, 256, 256, 256, 256, 1.0, *scales)
        rc = L.moe_create(d, 64, I, 4, 1e-6, ctypes.byref(w), 16, ctypes.byref(h))
        assert not h.value or rc == 0
        return rc
    assert create(d=2112) == -2 and create(I=1600) == -2
    assert create(scales=(None, 256)) == -1 and create(scales=(256, None)) == -1
    assert create(scales=(256, 264)) == -3
    h = ctypes.c_void_p(7)
    w = sb.MoeWeights(sb.MOE_MXFP4, 256, 256, 256, 256, 256, 1.0, 256, 256)
    assert L.moe_ep_create(2048, 64, 1536, 4, 1e-6, ctypes.byref(w), 16, 0, 8, 64,
                           ctypes.byref(h)) == -1
    assert L.moe_route_noalloc(256, sb.MOE_MXFP4, 256, 256, 256, 8, 256, 16, 4, 1e-6, 1.0, 256, 256,
                               None) == -1


def test_sizes_past_32_bits_are_refused():
    """Widths whose low 32 bits would look like a small one. The tensors have no
    storage: nothing is allocated and nothing launched."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    K = (1 << 32) + 128
    with FakeTensorMode():
        def q(*lead):
            return mx.MxTensor(*(torch.empty(*lead, K // d, dtype=torch.uint8, device="cuda:0")
                                 for d in (2, 32)))
        for shape in ((K,), (2, K)):
            with pytest.raises(ValueError, match="2\\^31"):
                mx.quantize(torch.empty(shape, dtype=torch.bfloat16, device="cuda:0"))
        with pytest.raises(ValueError, match="2\\^31"):
            mx.dequantize(q())
        with pytest.raises(ValueError, match="2\\^31"):
            mx.matmul(q(1), q(16))
