"""The MXFP4 product on CTA pairs over more K stages than its rings have slots, and
several items a pair: up to four stages a run's weights stay in shared memory and
the rows' ring of three wraps within an item; beyond, both rings wrap and weights
are loaded for every item. With the scales by TMA (K % 512 == 0) and by the warps.
Reference and tolerance as in test_gpu_mx.py; its products run in 64 bits."""
import numpy as np
import pytest
import torch

from sigmoid_bias_top_b200 import mx
from tests import mx_ref as R

pytestmark = pytest.mark.gpu
EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
COUNTS = [0, 1, 15, 190, 192, 193, 0, 383, 385, 700, 96, 31, 576, 577, 2, 208, 300, 0, 1000, 224]


def quantized(rows, K, seed):
    """Codes of every kind, scales that differ from block to block."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return mx.MxTensor(*(torch.randint(lo, hi, (*rows, K // d), generator=g, device="cuda",
                                       dtype=torch.uint8) for d, lo, hi in ((2, 0, 256), (32, 122, 128))))


def values(q):
    return torch.from_numpy(R.values(q.codes.cpu().numpy(), q.scales.cpu().numpy())).cuda()


def check(out, a, w, offs, silu, before=None):
    want, bound = R.matmul(values(a), values(w), offs, silu, EPS[out.dtype])
    got = out.double().cpu()
    used = ~torch.isnan(want)
    worst = ((got - want).abs() / bound)[used]
    assert worst.max() <= 1, float(worst.max())
    if before is not None:
        assert torch.equal(got[~used], before.double().cpu()[~used])


@pytest.mark.parametrize("silu,dtype", [(False, torch.bfloat16), (True, torch.bfloat16),
                                        (False, torch.float32), (True, torch.float32)])
@pytest.mark.parametrize("K", [1536, 2048, 1664, 1920, 2560, 2176, 3584, 6144])
def test_grouped(K, silu, dtype):
    offs = [int(v) for v in 5 + np.cumsum([0] + COUNTS)]
    rows, E, N = offs[-1] + 11, len(COUNTS), 1056       # 37 row tiles x 5 weight tiles
    a, w = quantized((rows,), K, K), quantized((E, N), K, K + 1)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    before = torch.randn(rows, N // 2 if silu else N, device="cuda").to(dtype)
    out = mx.matmul(a, w, off, silu_mul=silu, dtype=dtype, out=before.clone())
    check(out, a, w, offs, silu, before)
    for _ in range(3):
        assert torch.equal(out, mx.matmul(a, w, off, silu_mul=silu, dtype=dtype, out=before.clone()))
    assert mx.status() == 0


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("rows,K,N", [(1003, 2048, 2976), (3000, 2176, 4128), (769, 6144, 3104),
                                      (2500, 1664, 8224)])
def test_dense(rows, K, N, silu):
    a, w = quantized((rows,), K, K), quantized((N,), K, K + 1)
    out = mx.matmul(a, w, silu_mul=silu)
    check(out, a, mx.MxTensor(w.codes[None], w.scales[None]), [0, rows], silu)
    assert torch.equal(out, mx.matmul(a, w, silu_mul=silu)) and mx.status() == 0
