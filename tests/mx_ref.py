"""MXFP4 and the balance loss in 64 bits on the CPU, from their definitions
(include/mx.h, include/balance.h); shares no code with the package."""
import numpy as np
import torch

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x):
    """x [rows, K] float64 numpy (values of the stored type) -> codes, scales (uint8)."""
    rows, K = x.shape
    v = x.reshape(rows, K // 32, 32)
    amax = np.abs(v).max(-1)                       # NaN where the block holds one
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    e = np.floor(np.log2(safe)).astype(int)
    e = np.where(2.0 ** e > safe, e - 1, np.where(2.0 ** (e + 1) <= safe, e + 1, e))
    e = np.where(amax == 0, -127, np.maximum(e - 2, -127))
    q = np.where(bad[..., None], 0.0, v) / (2.0 ** e)[..., None]
    # nearest level, ties to the even code, everything above 6 to 6
    dist = np.abs(np.abs(q)[..., None] - LEVELS)
    low = dist.argmin(-1)                          # the lower of two equal distances
    tie = (low < 7) & (np.take_along_axis(dist, np.minimum(low + 1, 7)[..., None], -1)[..., 0]
                       == np.take_along_axis(dist, low[..., None], -1)[..., 0])
    code = np.where(tie & (low % 2 == 1), low + 1, low)
    code = code | np.where(np.signbit(v), 8, 0)
    code[bad] = 0
    code = code.reshape(rows, K).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def values(codes, scales):
    """uint8 numpy [..., K/2], [..., K/32] -> float64 [..., K]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127))
    return v * np.repeat(f, 32, -1)


def matmul(a, w, offsets, silu_mul, out_eps):
    """a [rows, K], w [E, N, K] float64 tensors; offsets list. Returns (out,
    bound): the product and how far an fp32 computation, rounded once with unit
    roundoff out_eps, may be from it; rows of no expert are NaN.

    Products of two E2M1 values are multiples of 1/4 below 37, so the 32 of a
    block pair (one scale) sum exactly in fp32; each of the K / 32 block sums
    and the few additions after it may be off by a unit in the last place of
    the sum of magnitudes S so far, 2^-23 S, doubled for a truncating adder."""
    rows, K = a.shape
    E, N, _ = w.shape
    NO = N // 2 if silu_mul else N
    out = torch.full((rows, NO), float("nan"), dtype=torch.float64)
    bound = torch.zeros(rows, NO, dtype=torch.float64)
    u = (K / 32 + 2) * 2.0 ** -22
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        if offsets[e + 1] <= offsets[e]:
            continue
        y, s = a[r] @ w[e].t(), a[r].abs() @ w[e].abs().t()
        err = u * s
        if silu_mul:
            g, up, eg, eu = y[:, :NO], y[:, NO:], err[:, :NO], err[:, NO:]
            y = g * torch.sigmoid(g) * up
            # |silu'| <= 1.1, |silu(g)| <= |g|; 2^-19 for the fast exponential
            # and division
            err = 1.1 * eg * (up.abs() + eu) + g.abs() * eu + 2.0 ** -19 * y.abs()
        out[r], bound[r] = y, err + out_eps * (y.abs() + err) + 1e-38
    return out, bound


def balance(logits, idx, offsets, coef, eps):
    """logits [n, E] float64 tensor; idx [n, k]; offsets list -> dict of float64
    (loss, counts, prob, grad), grad by the formula."""
    n, E = logits.shape
    k, B = idx.shape[1], len(offsets) - 1
    s = torch.sigmoid(logits)
    total = s.sum(1, keepdim=True) + eps
    p = torch.where(total > 0, s / total, torch.zeros_like(s))
    counts = torch.zeros(B, E, dtype=torch.float64)
    prob = torch.zeros(B, E, dtype=torch.float64)
    grad = torch.zeros(n, E, dtype=torch.float64)
    live = sum(offsets[b + 1] > offsets[b] for b in range(B))
    loss = 0.0
    for b in range(B):
        t0, t1 = offsets[b], offsets[b + 1]
        if t1 <= t0:
            continue
        sel = idx[t0:t1].flatten()
        for e in sel[(sel >= 0) & (sel < E)].tolist():
            counts[b, e] += 1
        prob[b] = p[t0:t1].mean(0)
        f = E * counts[b] / (k * (t1 - t0))
        loss = loss + coef / live * (f * prob[b]).sum()
        g = coef / live * f / (t1 - t0)
        pt, st = p[t0:t1], s[t0:t1]
        slope = torch.sigmoid(-logits[t0:t1]) * st
        inv = torch.where(total[t0:t1] > 0, 1 / total[t0:t1], torch.zeros(()).double())
        grad[t0:t1] = (g - (g * pt).sum(1, keepdim=True)) * inv * slope
    return {"loss": torch.as_tensor(loss), "counts": counts, "prob": prob, "grad": grad}
