"""ctypes binding of the router's balance loss (include/balance.h): argument
checks, autograd and marshalling only; the loss, the counts and the gradient
are computed by libmoe.so's CUDA kernels.

For router logits l [n, E] and the selected experts idx [n, k] (route_noalloc),
in the sequences b that seq_offsets cuts the tokens into, T_b tokens each:
  s = sigmoid(l),  p_te = s_te / (sum_j s_tj + eps)
  f_be = E counts_be / (k T_b),  prob_be = mean over b's tokens of p_te
  loss = coef * mean over the sequences with tokens of sum_e f_be prob_be
The counts carry no gradient; that of the logits runs through p.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import MOE_BF16, MOE_F32, _check, lib as _moe_lib
from .mx import _INT, _On, _here, _raw_stream

_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


class Balance(NamedTuple):
    loss: torch.Tensor     # [] f32, differentiable with respect to the logits
    counts: torch.Tensor   # [B, E] int32: slots of the sequence's tokens that hold the expert;
                           # the caller's to change (the gradient does not read it)
    prob: torch.Tensor     # [B, E] f32: mean normalised score (no gradient)


_bound = False


def lib():
    global _bound
    L = _moe_lib()
    if not _bound:
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        L.moe_balance_workspace.argtypes = [I, I, I]
        L.moe_balance_workspace.restype = ctypes.c_size_t
        L.moe_balance_forward.argtypes = [P, I, I64, P, P, I, I, I, I, F, F, P, P, P, P, P, P]
        L.moe_balance_forward.restype = I
        L.moe_balance_forward_kept.argtypes = L.moe_balance_forward.argtypes[:-1] + [P, P]
        L.moe_balance_forward_kept.restype = I
        L.moe_balance_backward.argtypes = [P, I, I64, P, P, P, P, I, I, I, I, F, P, P]
        L.moe_balance_backward.restype = I
        _bound = True
    return L


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ld(logits):
    """Elements from a row to the next (any, where there is no next)."""
    return logits.stride(0) if logits.shape[0] > 1 else logits.shape[1]


def _gradient(ctx, grad_loss):
    logits, kept, seq_offsets = ctx.saved_tensors
    n, E = logits.shape
    B, dev, counts = ctx.B, logits.device, kept.data_ptr()
    grad = logits.new_empty((n, E))
    # autograd runs this with the forward call's device and stream current
    _check(lib().moe_balance_backward(logits.data_ptr(), _DTYPES[logits.dtype], _ld(logits),
                                      counts, _ptr(seq_offsets), counts + 4 * B * E,
                                      grad_loss.data_ptr(), n, E, ctx.k, B, ctx.eps,
                                      grad.data_ptr(),
                                      _raw_stream(dev.index)), "moe_balance_backward")
    return grad


class _FirstOrder(torch.autograd.Function):
    """grad as it is, as a function of what it was computed from whose derivative is
    refused. A gradient without a graph would be a constant to a second
    differentiation, which would then leave it out of a sum with other losses'."""

    @staticmethod
    def forward(ctx, grad, logits, grad_loss):
        return grad

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("balance_loss has no second derivative")


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, idx, seq_offsets, coef, eps):
        n, E = logits.shape
        k, dev = idx.shape[1], logits.device
        B = 1 if seq_offsets is None else seq_offsets.numel() - 1
        L = lib()
        loss = logits.new_empty((), dtype=torch.float32)
        counts = idx.new_empty((B, E))
        # the backward pass's own counts (the caller may sum the others over ranks in
        # place, which autograd does not see) and behind them its scale
        kept = idx.new_empty(B * E + 1)
        prob = logits.new_empty((B, E), dtype=torch.float32)
        ws = idx.new_empty((L.moe_balance_workspace(n, E, B) + 3) // 4)
        own = kept.data_ptr()
        _check(L.moe_balance_forward_kept(logits.data_ptr(), _DTYPES[logits.dtype], _ld(logits),
                                          idx.data_ptr(), _ptr(seq_offsets), n, E, k, B, coef, eps,
                                          ws.data_ptr(), loss.data_ptr(), counts.data_ptr(),
                                          prob.data_ptr(), own + 4 * B * E, own,
                                          _raw_stream(dev.index)), "moe_balance_forward")
        ctx.save_for_backward(logits, kept, seq_offsets)
        ctx.B, ctx.k, ctx.eps = B, k, eps
        ctx.mark_non_differentiable(counts, prob)
        ctx.set_materialize_grads(False)
        return loss, counts, prob

    @staticmethod
    def backward(ctx, grad_loss, _counts, _prob):
        if grad_loss is None:
            return None, None, None, None, None
        grad = _gradient(ctx, grad_loss)
        if torch.is_grad_enabled():  # create_graph
            grad = _FirstOrder.apply(grad, ctx.saved_tensors[0], grad_loss)
        return grad, None, None, None, None


def balance_loss(logits, idx, seq_offsets: Optional[torch.Tensor] = None, coef: float = 1.0,
                 eps: float = 1e-6) -> Balance:
    """Balance loss, per-expert counts and mean scores of a routed batch.

    logits [n, E] f32 or bf16 (rows may be strided), idx [n, k] int32 (values
    outside [0, E) are dropped slots and not counted), seq_offsets [B + 1] int32
    on the device (None: one sequence of all tokens); tokens of no sequence take
    no part and get a zero gradient. There is no second derivative: asking for one
    raises RuntimeError. Runs on the current stream; the backward pass
    on the stream that autograd gives it. E <= 256, k <= min(E, 8).

    In a CUDA graph, capture the forward and the backward pass together, with no
    result of an eager call on the same leaves alive: autograd runs a leaf's last
    step on the stream that first used it, and such a stream is not captured."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _DTYPES:
        raise TypeError("logits must be a float32 or bfloat16 tensor")
    if logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be an [n, E] CUDA tensor")
    n, E = logits.shape
    device = logits.device
    if (idx.dtype != torch.int32 or idx.dim() != 2 or idx.shape[0] != n
            or not idx.is_contiguous() or idx.device != device):
        raise ValueError(f"idx must be a contiguous int32 ({n}, k) tensor on {device}")
    if seq_offsets is not None and (
            seq_offsets.dtype != torch.int32 or seq_offsets.dim() != 1 or seq_offsets.numel() < 2
            or not seq_offsets.is_contiguous() or seq_offsets.device != device):
        raise ValueError(f"seq_offsets must be a contiguous int32 (B + 1,) tensor on {device}")
    if max(n, E, idx.shape[1]) >= _INT or seq_offsets is not None and seq_offsets.numel() > _INT:
        raise ValueError("tokens, experts, slots and sequences must each be fewer than 2^31")
    if not _here(device, None):
        with _On(device, None):
            return balance_loss(logits, idx, seq_offsets, coef, eps)
    if E > 1 and logits.stride(1) != 1 or _ld(logits) < E:
        logits = logits.contiguous()
    return Balance(*_BalanceLoss.apply(logits, idx, seq_offsets, float(coef), float(eps)))
