"""ctypes binding of the microscaled 4-bit (MXFP4) operators (include/mx.h):
argument checks and marshalling only; every step runs in libmoe.so's CUDA
kernels.

Format: along a row, every 32 consecutive values share one E8M0 scale (a byte s
for 2^(s - 127), 255 for NaN), and each value is a 4-bit E2M1 code (0, 0.5, 1,
1.5, 2, 3, 4, 6 and their negatives) times its scale; two codes a byte, the
first in the low four bits.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import MOE_BF16, MOE_F32, _check, lib as _moe_lib

BLOCK = 32
_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


class MxTensor(NamedTuple):
    """Rows in MXFP4: codes [..., K/2] and scales [..., K/32], both uint8."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.codes.shape[-1] * 2)


_bound = False


def lib():
    global _bound
    L = _moe_lib()
    if not _bound:
        P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.moe_mx_quantize.argtypes = [P, I, I64, I, I64, P, P, P]
        L.moe_mx_dequantize.argtypes = [P, P, I64, I, P, I, P]
        L.moe_mx_matmul.argtypes = [P, P, P, P, P, I, I, I, I, I, P, I, P]
        L.moe_mx_status.argtypes = []
        for f in (L.moe_mx_quantize, L.moe_mx_dequantize, L.moe_mx_matmul,
                  L.moe_mx_status):
            f.restype = I
        _bound = True
    return L


class _On:
    """Makes the device of the tensors and the stream to launch on current (the
    given stream, or that device's current one), so that copies and outputs made
    inside belong to that stream too."""

    def __init__(self, device, stream):
        self.inner = None
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self.inner = torch.cuda.stream(stream)
        elif device.index != torch.cuda.current_device():
            self.inner = torch.cuda.device(device)
        self.device = device

    def __enter__(self):
        if self.inner is not None:
            self.inner.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


def _mx(name: str, q: MxTensor, dims) -> None:
    c, s = q
    for what, t in (("codes", c), ("scales", s)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda:
            raise TypeError(f"{name}.{what} must be a uint8 CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name}.{what} must be contiguous")
    if (c.dim() not in dims or c.shape[:-1] != s.shape[:-1] or c.shape[-1] != 16 * s.shape[-1]
            or c.device != s.device):
        raise ValueError(f"{name}: codes [..., K/2] and scales [..., K/32] of one shape and device, "
                         f"got {tuple(c.shape)} and {tuple(s.shape)}")


def _out(out: Optional[torch.Tensor], shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if (out.dtype != dtype or tuple(out.shape) != tuple(shape) or out.device != device
            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous {dtype} {tuple(shape)} tensor on {device}")
    return out


def quantize(x: torch.Tensor, out: Optional[MxTensor] = None, stream=None) -> MxTensor:
    """MXFP4 of x [..., K] (f32 or bf16, K % 32 == 0). A matrix may have strided
    rows; other layouts that the kernel cannot read in place are copied first."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError("x must be a float32 or bfloat16 tensor")
    if not x.is_cuda or x.dim() < 1 or x.shape[-1] == 0 or x.shape[-1] % BLOCK:
        raise ValueError("x must be a [..., K] CUDA tensor with K a multiple of 32")
    K = x.shape[-1]
    lead = tuple(x.shape[:-1])
    with _On(x.device, stream) as s:
        ld = K
        if not x.is_contiguous():
            if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= K and \
                    x.stride(0) * x.element_size() % 16 == 0:
                ld = x.stride(0)
            else:
                x = x.contiguous()
        if x.data_ptr() % 16:
            x, ld = x.clone(memory_format=torch.contiguous_format), K
        if out is None:
            out = MxTensor(torch.empty(*lead, K // 2, dtype=torch.uint8, device=x.device),
                           torch.empty(*lead, K // BLOCK, dtype=torch.uint8, device=x.device))
        else:
            out = MxTensor(_out(out[0], (*lead, K // 2), torch.uint8, x.device),
                           _out(out[1], (*lead, K // BLOCK), torch.uint8, x.device))
        _check(lib().moe_mx_quantize(x.data_ptr(), _DTYPES[x.dtype], x.numel() // K, K, ld,
                                     out.codes.data_ptr(), out.scales.data_ptr(), s),
               "moe_mx_quantize")
    return out


def dequantize(q: MxTensor, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """The values of q, [..., K] in dtype (bf16 holds those of quantize exactly)."""
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32 or bfloat16")
    _mx("q", q, range(1, 9))
    codes, scales = q
    K = codes.shape[-1] * 2
    if K == 0:
        raise ValueError("q has no columns")
    with _On(codes.device, stream) as s:
        out = _out(out, (*codes.shape[:-1], K), dtype, codes.device)
        _check(lib().moe_mx_dequantize(codes.data_ptr(), scales.data_ptr(), out.numel() // K, K,
                                       out.data_ptr(), _DTYPES[dtype], s), "moe_mx_dequantize")
    return out


def matmul(a: MxTensor, w: MxTensor, offsets: Optional[torch.Tensor] = None,
           silu_mul: bool = False, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """a [rows, K] times the transposes of quantised matrices.

    w [N, K] without offsets: one matrix for every row. w [E, N, K] with offsets
    [E + 1] (int32, on the device): rows offsets[e] .. offsets[e + 1] - 1 take
    matrix e; rows of no expert are left as they were (as allocated, without
    out). silu_mul: w holds the gate rows, then the up rows, and the result is
    silu(gate) * up, [rows, N / 2]. K % 128 == 0, N % 16 == 0 (32 with
    silu_mul), E <= 256. Sums are fp32, rounded once to dtype (bf16 or f32)."""
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32 or bfloat16")
    _mx("a", a, (2,))
    _mx("w", w, (2,) if offsets is None else (3,))
    rows, K = a.shape
    E = 1 if offsets is None else w.codes.shape[0]
    N = w.codes.shape[-2]
    if w.shape[-1] != K or w.codes.device != a.codes.device:
        raise ValueError(f"w must hold rows of {K} values on {a.codes.device}")
    if offsets is not None and (offsets.dtype != torch.int32 or tuple(offsets.shape) != (E + 1,)
                                or not offsets.is_contiguous()
                                or offsets.device != a.codes.device):
        raise ValueError(f"offsets must be a contiguous int32 ({E + 1},) tensor on "
                         f"{a.codes.device}")
    with _On(a.codes.device, stream) as s:
        out = _out(out, (rows, N // 2 if silu_mul else N), dtype, a.codes.device)
        _check(lib().moe_mx_matmul(a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(),
                                   w.scales.data_ptr(),
                                   None if offsets is None else offsets.data_ptr(), rows, K, E, N,
                                   int(silu_mul), out.data_ptr(), _DTYPES[dtype], s),
               "moe_mx_matmul")
    return out


def status(device=None) -> int:
    """Waits for the device; 0, or the code of a time-out inside a matmul on it
    since the last call (whose result is then incomplete)."""
    with torch.cuda.device(device):
        return lib().moe_mx_status()
