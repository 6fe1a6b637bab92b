"""MoE layers with MXFP4 experts, and the operators run together as a step uses
them: route, count and balance, quantise, the experts' two products, combine.

Reference: the layer in 64 bits on the GPU's own routing, with the two
quantisations of the forward done by the 64-bit quantiser on values rounded to
bf16 as the layer rounds them. What remains is fp32 summation order, the bf16
roundings of the expert outputs and of the result (2^-8 each), and codes that
round the other way because a bf16 input does: an fp32 value 2^-20 off rounds to
another bf16 with probability 2^-11, that to another code with 2^-6, so 0.01
codes of a row of 1536, each worth at most a third of one value, 1% of the row's
norm. Per token the MoE part may be 2e-2 off its norm, as for FP8 layers."""
import numpy as np
import pytest
import torch

import oracle
from sigmoid_bias_top_b200 import MoeError, MoeLayer, balance, mx, route_noalloc, workloads as W
from tests import mx_ref as R, parity as PA

pytestmark = pytest.mark.gpu
TOL, OUT_ROUND = 2e-2, 2.0 ** -8


def bf16(v):
    return torch.from_numpy(v).to(torch.bfloat16).double().numpy()


def quantized(v):
    return R.values(*R.quantize(bf16(v)))


def reference(x, layer, q, idx, k, eps, scale):
    """x + MoE part in float64 for the selection idx; experts from the codes q."""
    xd = x.double().cpu().numpy()
    gain = layer["norm_gain"].double().cpu().numpy()
    xn = xd / np.sqrt((xd ** 2).mean(1, keepdims=True) + eps) * gain
    s = 1 / (1 + np.exp(-(xn @ layer["router_w"].double().cpu().numpy().T)))
    sel = np.take_along_axis(s, idx, 1)
    w = scale * sel / (sel.sum(1, keepdims=True) + eps)
    xq = quantized(xn)
    out = np.zeros_like(xd)
    wgu, wd = ([q[n].cpu().numpy(), q[n + "_scale"].cpu().numpy()] for n in ("w_gate_up", "w_down"))
    I = wgu[0].shape[1] // 2
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        g = xq[t] @ R.values(wgu[0][e], wgu[1][e]).T
        act = g[:, :I] / (1 + np.exp(-g[:, :I])) * g[:, I:]
        y = quantized(act) @ R.values(wd[0][e], wd[1][e]).T
        out[t] += w[t, j][:, None] * y
    return xd + out, w


def check(out, x, ref):
    o, xd = out.double().cpu().numpy(), x.double().cpu().numpy()
    dn = np.maximum(np.linalg.norm(ref - xd, axis=1), 1e-30)
    err = np.linalg.norm(o - ref, axis=1)
    allowed = TOL * dn + OUT_ROUND * np.linalg.norm(ref, axis=1)
    assert np.all(err <= allowed), float((err / allowed).max())


def make(n, d, E, k, I, seed):
    w = W.DECODE.scaled(n_tokens=n, d=d, n_experts=E, top_k=k, d_ff=I, seed=seed, router_std=0.06,
                        gate_up_std=0.06, down_std=0.06)
    layer = W.make_layer(w, 0, "cuda")
    return w, layer, mx.quantize_experts(layer), W.make_x(w, "cuda")


@pytest.mark.parametrize("n,d,E,k,I", [(1, 256, 16, 4, 128), (33, 256, 16, 4, 384),
                                       (600, 384, 8, 2, 256), (64, 128, 64, 8, 128),
                                       (200, 512, 40, 1, 640)])
def test_layer_against_reference(n, d, E, k, I):
    w, layer, q, x = make(n, d, E, k, I, n)
    m = MoeLayer(q, k, w.eps, w.routed_scale, max_tokens=n)
    out = m(x)
    torch.cuda.synchronize()
    assert m.status() == 0 and m.launches_per_forward(n) == 7
    r = m.debug_routing(n)
    idx = r["idx"].cpu().numpy().astype(np.int64)
    PA.check_routing(x.cpu(), PA.to_cpu_layer(layer), k, w.eps, w.routed_scale, r)
    PA.check_dispatch(r["idx"].cpu().numpy(), E, r)
    ref, _ = reference(x, layer, q, idx, k, w.eps, w.routed_scale)
    check(out, x, ref)
    y = x.clone()
    m(y, y)                                   # in place, and the same bits again
    assert torch.equal(y, out)
    m.close()


def test_full_width_sampled_and_profiled():
    w = W.DECODE.scaled(n_tokens=96, seed=31)
    layer = W.make_layer(w, 0, "cuda")
    q = mx.quantize_experts(layer)
    x = W.make_x(w, "cuda")
    m = MoeLayer(q, w.top_k, w.eps, max_tokens=96)
    m.profile()
    out = m(x)
    assert list(m.kernel_times()) == ["route", "dispatch", "quantize", "gate_up", "quantize_act",
                                      "down", "combine"]
    m.profile(False)
    idx = m.debug_routing(96)["idx"].cpu().numpy().astype(np.int64)
    toks = np.arange(0, 96, 8)
    ref, _ = reference(x[::8], layer, q, idx[toks], w.top_k, w.eps, 1.0)
    check(out[::8], x[::8], ref)
    host = torch.empty_like(x, device="cpu").pin_memory()
    m.forward_host(x.cpu().pin_memory(), host)
    assert torch.equal(host, out.cpu())
    m.close()


def test_captured_forward():
    w, layer, q, x = make(50, 256, 16, 4, 256, 3)
    m = MoeLayer(q, 4, w.eps, max_tokens=50)
    want = [m(x), m(-2 * x)]
    out = torch.empty_like(x)
    xs = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m(xs, out)
    for scale, ref in ((1, want[0]), (-2, want[1])):
        xs.copy_(scale * x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    m.close()


@pytest.mark.parametrize("n", [40, 700])
def test_the_operators_give_the_layers_result(n):
    """A step built from the public operators: the router's selection, its counts
    (whose running sums are the groups' offsets), rows quantised, both products
    and the weighted sum, against the layer's own forward; and the balance loss
    of the same selection."""
    d, E, k, I = 256, 16, 4, 384
    w, layer, q, x = make(n, d, E, k, I, 5)
    idx, wts = route_noalloc(x, layer, k, w.eps)
    xf = x.float()
    xn = xf * torch.rsqrt((xf * xf).mean(1, keepdim=True) + w.eps) * layer["norm_gain"]
    logits = (xn @ layer["router_w"].t()).requires_grad_()
    b = balance.balance_loss(logits, idx, torch.tensor([0, n // 3, n], dtype=torch.int32, device="cuda"),
                             coef=0.01)
    b.loss.backward()
    ref = R.balance(logits.detach().double().cpu(), idx.cpu(), [0, n // 3, n], 0.01, 1e-6)
    assert torch.equal(b.counts.cpu().double(), ref["counts"])
    torch.testing.assert_close(b.loss.detach().double().cpu(), ref["loss"], rtol=1e-4, atol=0)
    torch.testing.assert_close(logits.grad.double().cpu(), ref["grad"], rtol=1e-3,
                               atol=1e-4 * float(ref["grad"].abs().max()))

    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = b.counts.sum(0).cumsum(0)
    order = torch.sort(idx.flatten().long(), stable=True).indices      # grouped by expert
    rows = mx.quantize(xn.bfloat16()[order // k])
    experts = [mx.MxTensor(q[name], q[name + "_scale"]) for name in ("w_gate_up", "w_down")]
    act = mx.matmul(rows, experts[0], offsets, silu_mul=True)
    y = mx.matmul(mx.quantize(act), experts[1], offsets)
    out = xf.clone()
    out.index_add_(0, order // k, y.float() * wts.flatten()[order, None])
    assert mx.status() == 0

    m = MoeLayer(q, k, w.eps, max_tokens=n)
    assert torch.equal(m.debug_routing(0)["offsets"][:1], offsets[:1])
    own = m(x)
    assert torch.equal(m.debug_routing(n)["offsets"], offsets)
    full, _ = reference(x, layer, q, idx.cpu().numpy().astype(np.int64), k, w.eps, 1.0)
    check(out, x, full)
    check(own, x, full)
    m.close()


def test_refusals():
    w, layer, q, x = make(4, 256, 16, 4, 128, 1)
    bad = dict(q, w_down_scale=q["w_down_scale"][:, :, :1].contiguous())
    with pytest.raises(ValueError):
        MoeLayer(bad, 4, w.eps)
    with pytest.raises(ValueError):
        mx.quantize_experts(W.make_layer(w.scaled(d_ff=192), 0, "cuda"))
    m = MoeLayer(q, 4, w.eps, max_tokens=4)
    with pytest.raises(MoeError):
        m(W.make_x(w.scaled(n_tokens=5), "cuda"))
    with pytest.raises(MoeError):
        m.debug_fp8_rows(0)
    m.close()
