"""The MXFP4 and balance bindings with a torch that lacks the functions behind
their fast lookups of the current device and stream, as a torch without CUDA."""
import subprocess
import sys

CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from sigmoid_bias_top_b200 import balance, mx
for call, error in ((lambda: mx.quantize(torch.zeros(4, 64)), ValueError),
                    (lambda: mx.quantize(torch.zeros(4, 64).half()), TypeError),
                    (lambda: balance.balance_loss(torch.zeros(4, 8),
                                                  torch.zeros(4, 2, dtype=torch.int32)), ValueError)):
    try:
        call()
    except error:
        continue
    raise SystemExit("not refused")

class Stream:
    cuda_stream = 7
torch.cuda.current_stream = lambda device: Stream if device == 3 else None
torch.cuda.current_device = lambda: 3
assert mx._raw_stream(3) == 7 and mx._current_device() == 3
"""


def test_import_and_refusals_without_them():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
