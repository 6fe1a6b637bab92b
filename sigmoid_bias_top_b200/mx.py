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
_INT = 1 << 31  # sizes pass as C ints, of which ctypes keeps the low 32 bits without a word
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
        L.moe_mx_selftest_timeout.argtypes = [P, P, P, P, P, I, I, I, I, I, P, I, I, I, P]
        L.moe_mx_status.argtypes = []
        for f in (L.moe_mx_quantize, L.moe_mx_dequantize, L.moe_mx_matmul,
                  L.moe_mx_selftest_timeout, L.moe_mx_status):
            f.restype = I
        _bound = True
    return L


# The current device, and the current stream's handle on a device without building a
# Stream; the public functions where torch has no such ones.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda index: torch.cuda.current_stream(index).cuda_stream))


class _On:
    """Makes the device of the tensors and the stream to launch on current (the
    given stream, or that device's current one), so that copies and outputs made
    inside belong to that stream too. Only needed where _here says no. A stream that
    was given is recorded as a user of the tensors: the memory of those dropped
    after the call is not handed out again before the stream is done with them."""

    def __init__(self, device, stream, *tensors):
        if stream is None:
            self.inner = torch.cuda.device(device)
        else:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self.inner = torch.cuda.stream(stream)
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        self.inner.__enter__()

    def __exit__(self, *exc):
        self.inner.__exit__(*exc)


def _here(device, stream) -> bool:
    """Whether a launch needs neither another device nor another stream."""
    return stream is None and device.index == _current_device()


def _mx(name: str, q: MxTensor, least: int, most: int):
    """Checks a quantised argument; returns (codes, scales, its device)."""
    c, s = q
    for what, t in (("codes", c), ("scales", s)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda:
            raise TypeError(f"{name}.{what} must be a uint8 CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name}.{what} must be contiguous")
    cs, ss = c.shape, s.shape
    device = c.device
    if (not least <= len(cs) <= most or cs[:-1] != ss[:-1] or cs[-1] != 16 * ss[-1]
            or device != s.device):
        raise ValueError(f"{name}: codes [..., K/2] and scales [..., K/32] of one shape and device, "
                         f"got {tuple(cs)} and {tuple(ss)}")
    if 2 * cs[-1] >= _INT:
        raise ValueError(f"{name}: rows of fewer than 2^31 values, got {2 * cs[-1]}")
    return c, s, device


def _out(out: Optional[torch.Tensor], shape, dtype, device):
    """Checks an output that the caller gave."""
    if (out.dtype != dtype or tuple(out.shape) != tuple(shape) or out.device != device
            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous {dtype} {tuple(shape)} tensor on {device}")
    return out


def quantize(x: torch.Tensor, out: Optional[MxTensor] = None, stream=None) -> MxTensor:
    """MXFP4 of x [..., K] (f32 or bf16, K % 32 == 0). A matrix may have strided
    rows; other layouts that the kernel cannot read in place are copied first."""
    dt = _DTYPES.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if dt is None:
        raise TypeError("x must be a float32 or bfloat16 tensor")
    shape = x.shape
    if not x.is_cuda or len(shape) < 1 or shape[-1] == 0 or shape[-1] % BLOCK:
        raise ValueError("x must be a [..., K] CUDA tensor with K a multiple of 32")
    if shape[-1] >= _INT:
        raise ValueError(f"x must have rows of fewer than 2^31 values, got {shape[-1]}")
    device = x.device
    if not _here(device, stream):
        with _On(device, stream, x, *(out or ())):
            return quantize(x, out)
    K = ld = shape[-1]
    if not x.is_contiguous():
        if len(shape) == 2 and x.stride(1) == 1 and x.stride(0) >= K and \
                x.stride(0) * x.element_size() % 16 == 0:
            ld = x.stride(0)
        else:
            x = x.contiguous()
    ptr = x.data_ptr()
    if ptr % 16:
        x, ld = x.clone(memory_format=torch.contiguous_format), K
        ptr = x.data_ptr()
    lead = shape[:-1]
    if out is None:
        codes = x.new_empty((*lead, K // 2), dtype=torch.uint8)
        scales = x.new_empty((*lead, K // BLOCK), dtype=torch.uint8)
    else:
        codes = _out(out[0], (*lead, K // 2), torch.uint8, device)
        scales = _out(out[1], (*lead, K // BLOCK), torch.uint8, device)
    _check(lib().moe_mx_quantize(ptr, dt, x.numel() // K, K, ld, codes.data_ptr(),
                                 scales.data_ptr(), _raw_stream(device.index)), "moe_mx_quantize")
    return MxTensor(codes, scales)


def dequantize(q: MxTensor, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """The values of q, [..., K] in dtype (bf16 holds those of quantize exactly)."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("dtype must be float32 or bfloat16")
    codes, scales, device = _mx("q", q, 1, 8)
    shape = codes.shape
    K = shape[-1] * 2
    if K == 0:
        raise ValueError("q has no columns")
    if not _here(device, stream):
        with _On(device, stream, codes, scales, out):
            return dequantize(q, dtype, out)
    if out is None:
        out = codes.new_empty((*shape[:-1], K), dtype=dtype)
    else:
        _out(out, (*shape[:-1], K), dtype, device)
    _check(lib().moe_mx_dequantize(codes.data_ptr(), scales.data_ptr(), out.numel() // K, K,
                                   out.data_ptr(), dt, _raw_stream(device.index)),
           "moe_mx_dequantize")
    return out


def matmul(a: MxTensor, w: MxTensor, offsets: Optional[torch.Tensor] = None,
           silu_mul: bool = False, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """a [rows, K] times the transposes of quantised matrices.

    w [N, K] without offsets: one matrix for every row. w [E, N, K] with offsets
    [E + 1] (int32, on the device): rows offsets[e] .. offsets[e + 1] - 1 take
    matrix e; rows of no expert are left as they were (as allocated, without
    out). silu_mul: w holds the gate rows, then the up rows, and the result is
    silu(gate) * up, [rows, N / 2]. K % 128 == 0, K <= 2^22, N % 16 == 0
    (32 with silu_mul), E <= 256. Sums are fp32, rounded once to dtype (bf16 or f32)."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("dtype must be float32 or bfloat16")
    ac, as_, device = _mx("a", a, 2, 2)
    wc, ws, w_device = _mx("w", w, 2, 2) if offsets is None else _mx("w", w, 3, 3)
    rows, half = ac.shape
    N = wc.shape[-2]
    if rows >= _INT or N >= _INT:
        raise ValueError(f"fewer than 2^31 rows, got {rows} of a and {N} of w")
    if wc.shape[-1] != half or w_device != device:
        raise ValueError(f"w must hold rows of {2 * half} values on {device}")
    E, offs = 1, None
    if offsets is not None:
        E = wc.shape[0]
        if (offsets.dtype != torch.int32 or tuple(offsets.shape) != (E + 1,)
                or not offsets.is_contiguous() or offsets.device != device):
            raise ValueError(f"offsets must be a contiguous int32 ({E + 1},) tensor on {device}")
        offs = offsets.data_ptr()
    if not _here(device, stream):
        with _On(device, stream, ac, as_, wc, ws, offsets, out):
            return matmul(a, w, offsets, silu_mul, dtype, out)
    if out is None:
        out = ac.new_empty((rows, N // 2 if silu_mul else N), dtype=dtype)
    else:
        _out(out, (rows, N // 2 if silu_mul else N), dtype, device)
    _check(lib().moe_mx_matmul(ac.data_ptr(), as_.data_ptr(), wc.data_ptr(), ws.data_ptr(), offs,
                               rows, 2 * half, E, N, 1 if silu_mul else 0, out.data_ptr(), dt,
                               _raw_stream(device.index)), "moe_mx_matmul")
    return out


def quantize_experts(layer):
    """A MoeLayer dict with its expert matrices (f32 or bf16) in MXFP4: codes under
    w_gate_up and w_down, scales under w_gate_up_scale and w_down_scale; the rest
    as it was. Widths must be multiples of 128."""
    out = dict(layer)
    for name in ("w_gate_up", "w_down"):
        if layer[name].shape[-1] % 128:
            raise ValueError(f"{name}: rows of a multiple of 128 values")
        out[name], out[name + "_scale"] = quantize(layer[name])
    return out


def status(device=None) -> int:
    """Waits for the device; 0, or the code of a time-out inside a matmul on it, by any
    thread, since this thread's last call (the result is then incomplete). Every
    thread that asks is told."""
    with torch.cuda.device(device):
        return lib().moe_mx_status()
