"""Several threads whose first MXFP4 products come at once, in a process of their
own: what a kernel's first launch sets up is set up once, and every thread gets
the same bits."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
CODE = """
import threading, torch
from sigmoid_bias_top_b200 import mx
torch.manual_seed(0)
a = mx.quantize(torch.randn(1500, 512, device="cuda"))
w = mx.quantize(torch.randn(2304, 512, device="cuda"))
few = mx.MxTensor(a.codes[:9], a.scales[:9])
torch.cuda.synchronize()
n, outs = 8, [None] * 8
gate = threading.Barrier(n)
def run(i):
    s = torch.cuda.Stream()
    gate.wait()
    pair = [mx.matmul(q, w, silu_mul=silu, stream=s) for q in (a, few) for silu in (False, True)]
    s.synchronize()
    outs[i] = pair
threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
for o in outs:
    assert o is not None and all(torch.equal(x, y) for x, y in zip(o, outs[0]))
for x, q, silu in zip(outs[0], (a, a, few, few), (False, True) * 2):
    assert torch.equal(x, mx.matmul(q, w, silu_mul=silu))
assert mx.status() == 0
"""


def test_first_products_of_several_threads():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
