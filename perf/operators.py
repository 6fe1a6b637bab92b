"""Measured cases of the 4-bit (MXFP4) quantiser and product and of the router's
balance loss.

Every case is one call that a program makes: "quantize" brings rows to MXFP4 and
back to the values that the codes stand for, "matmul" multiplies quantised rows
by the quantised matrices of their experts (or of one dense layer), "balance"
is the router's balance loss with its per-expert counts and the gradient of the
logits. `run` computes them from elementary torch operations, or with `own` set
by the package's kernels; `exact` computes them in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32                       # values per shared scale
ZIPF = 1.2                       # load exponent of the skewed expert groups


# ---------------------------------------------------------------------------
# Cases

def listed():
    """Width 2048, 64 experts of width 1536 with four a token, and the dense
    block's 6144 are this repository's workloads."""
    return [
        # the grouped rows of one decode step: 32 tokens, four experts each
        {"name": "quantize decode rows", "op": "quantize", "rows": 128, "k": 2048, "dtype": "bf16"},
        # the same of a prefill of 8192 tokens
        {"name": "quantize prefill rows", "op": "quantize", "rows": 32768, "k": 2048,
         "dtype": "bf16"},
        # an odd number of fp32 rows of an expert's inner width
        {"name": "quantize odd f32 rows", "op": "quantize", "rows": 4099, "k": 1536, "dtype": "f32"},
        # decode: the experts' two products, bound by the weights' stream
        {"name": "experts gate/up decode", "op": "matmul", "rows": 128, "k": 2048, "n": 1536,
         "experts": 64, "load": "uniform", "silu": True},
        {"name": "experts down decode", "op": "matmul", "rows": 128, "k": 1536, "n": 2048,
         "experts": 64, "load": "uniform", "silu": False},
        # one token through a dense layer
        {"name": "dense one token", "op": "matmul", "rows": 1, "k": 2048, "n": 2048,
         "experts": 0, "load": "uniform", "silu": False},
        # prefill: 8192 tokens, near-uniform load
        {"name": "experts gate/up prefill", "op": "matmul", "rows": 32768, "k": 2048, "n": 1536,
         "experts": 64, "load": "uniform", "silu": True},
        # 16384 tokens under a skewed load: some experts large, some nearly empty
        {"name": "experts down skewed", "op": "matmul", "rows": 65536, "k": 1536, "n": 2048,
         "experts": 64, "load": "zipf", "silu": False},
        # the dense block's down projection over 4 x 2048 positions
        {"name": "dense down prefill", "op": "matmul", "rows": 8192, "k": 6144, "n": 2048,
         "experts": 0, "load": "uniform", "silu": False},
        # a small training step: 64 tokens of 16 experts in ragged sequences
        {"name": "balance small", "op": "balance", "tokens": 64, "experts": 16, "top_k": 4,
         "seqs": 5, "dtype": "f32"},
        # 4 x 2048 positions, 64 experts, bf16 logits
        {"name": "balance 4 sequences", "op": "balance", "tokens": 8192, "experts": 64, "top_k": 4,
         "seqs": 4, "dtype": "bf16"},
        # a large batch over many experts, packed sequences of uneven lengths
        {"name": "balance large", "op": "balance", "tokens": 131072, "experts": 256, "top_k": 8,
         "seqs": 61, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "matmul", "matmul", "balance"))
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 32768), "k": BLOCK * _log_int(rng, 1, 64),
                "dtype": rng.choice(("bf16", "f32"))}
    if op == "matmul":
        e = rng.choice((0, 0, 2, 8, 16, 33, 64))
        k, n = 128 * _log_int(rng, 1, 16), 16 * _log_int(rng, 1, 96)
        if e == 0 and rng.random() < 0.5:
            k, n = 128 * _log_int(rng, 8, 48), 16 * _log_int(rng, 32, 256)
        most = 65536 * 1536 * 2048 // (k * n * 2)
        return {"op": op, "rows": _log_int(rng, 1, min(65536, most)), "k": k, "n": n, "experts": e,
                "load": rng.choice(("uniform", "zipf", "half")), "silu": rng.random() < 0.5}
    e = rng.choice((8, 16, 40, 64, 128, 256))
    t = _log_int(rng, 1, 131072)
    return {"op": op, "tokens": t, "experts": e, "top_k": rng.randint(1, 8),
            "seqs": _log_int(rng, 1, min(t, 256)), "dtype": rng.choice(("bf16", "f32"))}


# ---------------------------------------------------------------------------
# Inputs

def _loads(case):
    """Share of the rows that each expert group gets."""
    e = max(1, case["experts"])
    if case["load"] == "zipf":
        p = [1.0 / (r + 1) ** ZIPF for r in range(e)]
    elif case["load"] == "half":      # every other expert is without rows
        p = [1.0 if r % 2 == 0 else 0.0 for r in range(e)]
    else:
        p = [1.0] * e
    s = sum(p)
    return [v / s for v in p]


def _codes(shape, std, g):
    """N(0, std) values as MXFP4 (codes, scales), without any rounding subtlety:
    these are inputs, made block by block so that large matrices fit."""
    rows, k = shape
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, k // BLOCK, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // k)
    for r in range(0, rows, step):
        v = torch.randn(min(step, rows - r), k, generator=g, device="cuda") * std
        v = v.view(v.shape[0], -1, BLOCK)
        s = (v.abs().amax(-1).view(torch.int32) >> 23) - 2
        q = v.abs() * ((254 - s) << 23).view(torch.float32)[..., None]
        c = torch.bucketize(q, torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.], device="cuda"),
                            out_int32=True)
        c = (c + 8 * (v < 0)).to(torch.uint8).view(v.shape[0], k // 2, 2)
        codes[r:r + step] = c[..., 0] | (c[..., 1] << 4)
        scales[r:r + step] = s.to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    h = torch.Generator()
    h.manual_seed(int(seed))
    if case["op"] == "quantize":
        # normalised rows with a few large channels
        x = torch.randn(case["rows"], case["k"], generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(case["k"], generator=g, device="cuda"))
        return {"case": case, "x": x.to(DTYPES[case["dtype"]])}
    if case["op"] == "matmul":
        e, rows, k = max(1, case["experts"]), case["rows"], case["k"]
        n = case["n"] * (2 if case["silu"] else 1)
        a = _codes((rows, k), 1.0, g)
        w = _codes((e * n, k), 0.5 / math.sqrt(k) if not case["silu"] else 1 / math.sqrt(k), g)
        w = tuple(t.view(e, n, -1) for t in w) if case["experts"] else w
        off = None
        if case["experts"]:
            pick = torch.multinomial(torch.tensor(_loads(case)), rows, True, generator=h)
            off = torch.zeros(e + 1, dtype=torch.int32)
            off[1:] = torch.bincount(pick, minlength=e).cumsum(0)
            off = off.cuda()
        return {"case": case, "a": a, "w": w, "offsets": off}
    t, e, k, b = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    logits = torch.randn(t, e, generator=g, device="cuda")
    logits = (logits + 0.5 * torch.randn(e, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    # the router's selection: scores plus a stored bias
    bias = 0.05 * torch.randn(e, generator=g, device="cuda")
    idx = (torch.sigmoid(logits.float()) + bias).topk(min(k, e), 1).indices.to(torch.int32)
    cuts = torch.sort(torch.randint(0, t + 1, (b - 1,), generator=h)).values
    off = torch.cat([torch.tensor([0]), cuts, torch.tensor([t])]).to(torch.int32).cuda()
    return {"case": case, "logits": logits.requires_grad_(), "idx": idx, "offsets": off,
            "coef": 1e-2, "eps": 1e-6}


# ---------------------------------------------------------------------------
# The plain forms

def _value_pairs():
    """[256, 2] values of the two codes of a byte, the low four bits first."""
    v = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6.], device="cuda")
    v = torch.cat([v, -v])
    b = torch.arange(256, device="cuda")
    return torch.stack([v[b & 15], v[b >> 4]], 1)


def _values(codes, scales):
    v = _value_pairs()[codes.int()].view(*scales.shape, BLOCK)
    return (v * torch.ldexp(torch.ones((), device="cuda"), scales.int() - 127)[..., None]).flatten(-2)


def _plain_quantize(x):
    v = x.float().view(x.shape[0], -1, BLOCK)
    amax = v.abs().amax(-1)
    # shared exponent: that of the largest value, less the 2 of the largest code's
    e = ((amax.view(torch.int32) >> 23) - 127 - 2).clamp_min(-127)[..., None]
    q = torch.ldexp(v, -e)
    # a code's step is half the power of two at or below it, 0.5 under one
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0))
    q = (torch.round(q / step) * step).clamp(-6.0, 6.0)
    return torch.ldexp(q, e).view(x.shape).to(x.dtype)


def _plain_matmul(case, a, w, offsets):
    a, w = _values(*a), _values(*w)
    if offsets is None:
        y = a @ w.t()
    else:
        # rows in tiles that hold one expert's rows each
        rows, e = a.shape[0], w.shape[0]
        t = 16 if rows <= 16 * e else 128
        tiles = (offsets[1:] - offsets[:-1] + t - 1) // t
        first = torch.cumsum(tiles, 0) - tiles
        i = torch.arange(rows // t + e, device="cuda", dtype=torch.int32)
        g = (torch.searchsorted(first, i, right=True) - 1)
        g = torch.clamp(g, 0, e - 1)
        r = (offsets[g] + (i - first[g]) * t)[:, None] + torch.arange(t, device="cuda")
        r = torch.where((r < offsets[g + 1][:, None]) & (i < tiles.sum())[:, None], r, rows)
        y = torch.bmm(torch.cat([a, a.new_zeros(1, a.shape[1])])[r], w[g].transpose(1, 2))
        out = y.new_zeros(rows + 1, y.shape[-1])
        out[r.flatten()] = y.flatten(0, 1)
        y = out[:rows]
    if case["silu"]:
        gate, up = y[:, :case["n"]], y[:, case["n"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(torch.bfloat16)


def _plain_balance(logits, idx, offsets, coef, eps):
    l = logits.detach().float()
    n, e = l.shape
    k, b = idx.shape[1], offsets.numel() - 1
    s = 1 / (1 + torch.exp(-l))
    total = s.sum(1, keepdim=True) + eps
    p = s / total
    seq = torch.searchsorted(offsets, torch.arange(n, device="cuda", dtype=torch.int32),
                             right=True) - 1
    chosen = (idx[:, :, None] == torch.arange(e, device="cuda", dtype=torch.int32)).sum(1)
    counts = torch.zeros(b, e, device="cuda", dtype=torch.int64).index_add_(0, seq, chosen)
    length = (offsets[1:] - offsets[:-1]).clamp_min(1).float()[:, None]
    prob = torch.zeros(b, e, device="cuda", dtype=torch.float64).index_add_(0, seq, p.double())
    prob = (prob / length).float()
    share = counts.float() * (e / k) / length
    live = (offsets[1:] > offsets[:-1]).sum()
    loss = coef / live * (share * prob).double().sum()
    # counts have no gradient: d loss / d p = coef share / (live length)
    gp = (coef / live * share / length)[seq]
    grad = (gp - (gp * p).sum(1, keepdim=True)) / total * s * (1 - s)
    return {"loss": loss.float(), "counts": counts.int(), "prob": prob,
            "grad": grad.to(logits.dtype)}


def run(state):
    case = state["case"]
    if own:
        from sigmoid_bias_top_b200 import balance, mx
        if case["op"] == "quantize":
            return mx.dequantize(mx.quantize(state["x"]), state["x"].dtype)
        if case["op"] == "matmul":
            return mx.matmul(mx.MxTensor(*state["a"]), mx.MxTensor(*state["w"]),
                             offsets=state["offsets"], silu_mul=case["silu"])
        r = balance.balance_loss(state["logits"], state["idx"], state["offsets"],
                                 coef=state["coef"], eps=state["eps"])
        grad, = torch.autograd.grad(r.loss, state["logits"])
        return {"loss": r.loss.detach(), "counts": r.counts, "prob": r.prob, "grad": grad}
    if case["op"] == "quantize":
        return _plain_quantize(state["x"])
    if case["op"] == "matmul":
        return _plain_matmul(case, state["a"], state["w"], state["offsets"])
    return _plain_balance(state["logits"], state["idx"], state["offsets"], state["coef"],
                          state["eps"])


# ---------------------------------------------------------------------------
# Work and 64-bit results

def work(case):
    if case["op"] == "quantize":
        v = case["rows"] * case["k"]
        # x read, the codes with their scales written, the values written
        return {"bytes": v * (2 * DTYPES[case["dtype"]].itemsize + 0.5 + 1 / BLOCK), "flops": 0}
    if case["op"] == "matmul":
        n = case["n"] * (2 if case["silu"] else 1)
        rows, k = case["rows"], case["k"]
        live = sum(1 - (1 - p) ** rows for p in _loads(case))     # experts that have rows
        return {"bytes": (rows + live * n) * k * (0.5 + 1 / BLOCK) + rows * case["n"] * 2,
                "flops": 2 * rows * n * k}
    t, e, k, b = case["tokens"], case["experts"], min(case["top_k"], case["experts"]), case["seqs"]
    # logits read and their gradient written, the indices read; counts and shares
    return {"bytes": t * (2 * e * DTYPES[case["dtype"]].itemsize + 4 * k) + 8 * b * e, "flops": 0}


def _exact_values(q):
    codes, scales = q
    table = torch.tensor([(-1.0) ** (c >> 3) * (0.5 * (c & 1) if (c >> 1) & 3 == 0 else
                          (1 + 0.5 * (c & 1)) * 2.0 ** (((c >> 1) & 3) - 1)) for c in range(16)],
                         dtype=torch.float64, device="cuda")
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def _exact_quantize(x):
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for r in range(0, x.shape[0], 4096):
        v = x[r:r + 4096].double().unflatten(1, (-1, BLOCK))
        m, e = torch.frexp(v.abs().amax(-1, keepdim=True))
        scale = torch.exp2(torch.where(m > 0, e - 3, -127).clamp_min(-127).double())
        q = (v / scale).abs()
        # how many of the midpoints lie below: ties go to the even code
        c = sum((q >= m if i % 2 else q > m).long()
                for i, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        out[r:r + 4096] = (torch.copysign(table[c], v) * scale).flatten(1)
    return out


def _exact_matmul(case, state):
    a, w, off = state["a"], state["w"], state["offsets"]
    cuts = [0, case["rows"]] if off is None else off.tolist()
    w = tuple(t if t.dim() == 3 else t[None] for t in w)
    out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
    for i in range(len(cuts) - 1):
        if cuts[i + 1] > cuts[i]:
            m = _exact_values((w[0][i], w[1][i]))
            for r in range(cuts[i], cuts[i + 1], 8192):
                stop = min(cuts[i + 1], r + 8192)
                y = _exact_values((a[0][r:stop], a[1][r:stop])) @ m.t()
                if case["silu"]:
                    y = y[:, :case["n"]] * torch.sigmoid(y[:, :case["n"]]) * y[:, case["n"]:]
                out[r:stop] = y
    return out


def _exact_balance(state):
    off = state["offsets"].tolist()
    logits = state["logits"].detach().double().requires_grad_()
    n, e = logits.shape
    k = state["idx"].shape[1]
    score = torch.sigmoid(logits)
    p = score / (score.sum(1, keepdim=True) + state["eps"])
    live = [b for b in range(len(off) - 1) if off[b + 1] > off[b]]
    counts = torch.zeros(len(off) - 1, e, dtype=torch.int64, device="cuda")
    prob = torch.zeros(len(off) - 1, e, dtype=torch.float64, device="cuda")
    loss = 0.0
    for b in live:
        rows = slice(off[b], off[b + 1])
        counts[b] = torch.bincount(state["idx"][rows].flatten().long(), minlength=e)
        mean = p[rows].mean(0)
        prob[b] = mean.detach()
        loss = loss + (e / (k * (off[b + 1] - off[b])) * counts[b] * mean).sum()
    loss = state["coef"] / len(live) * loss
    grad, = torch.autograd.grad(loss, logits)
    return {"loss": loss.detach(), "counts": counts.int(), "prob": prob, "grad": grad}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(state["x"])
    if case["op"] == "matmul":
        return _exact_matmul(case, state)
    return _exact_balance(state)
