"""MXFP4 quantiser, its inverse and the product on the GPU against the 64-bit
reference. Quantising and dequantising are exact: codes, scales and values are
compared for equality. The product's tolerance is that of an fp32 sum rounded
once (derived at tests/mx_ref.py's matmul)."""
import numpy as np
import pytest
import torch

from sigmoid_bias_top_b200 import MoeError, mx
from tests import mx_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def check_quantized(q, x):
    codes, scales = R.quantize(x.double().cpu().numpy())
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)


# ------------------------------------------------------------------ quantise
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 32), (1, 2048), (5, 96), (31, 1056), (257, 1536),
                                    (1000, 2048)])
def test_quantize_rows(rows, K, dtype):
    x = (torch.randn(rows, K, generator=gen(rows + K), device="cuda") *
         torch.exp(3 * torch.randn(rows, 1, generator=gen(1), device="cuda"))).to(DT[dtype])
    q = mx.quantize(x)
    check_quantized(q, x)
    for out in ("bf16", "f32"):
        v = mx.dequantize(q, DT[out])
        assert v.dtype == DT[out]
        np.testing.assert_array_equal(
            v.double().cpu().numpy(), R.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_special_values(dtype):
    """Zeros, subnormals, the largest numbers, infinities, NaN, ties, saturation,
    one block each; neighbours of a bad block are untouched."""
    big = torch.finfo(DT[dtype]).max
    x = torch.zeros(12, 64, dtype=torch.float64)
    x[1, :] = 2.0 ** -133                      # a subnormal of both types
    x[2, 0], x[2, 33] = big, -big
    x[3, 5], x[3, 40] = float("inf"), 1.0
    x[4, 63], x[4, 0] = float("nan"), 3.0
    x[5, 7] = -float("inf")
    x[6] = torch.linspace(-8, 8, 64)
    x[7, :8] = torch.tensor([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.])
    x[8, :8] = -x[7, :8] * 2.0 ** -126         # scales at the lower end
    x[9] = -0.0
    x[10, 0], x[10, 1] = 2.0 ** -125, 2.0 ** -126
    x[11, 0], x[11, 1] = 2.0 ** 100, 2.0 ** 90
    x = x.to(DT[dtype])
    q = mx.quantize(x.cuda())
    check_quantized(q, x)
    v = mx.dequantize(q, torch.float32).cpu()
    assert torch.isnan(v[3, :32]).all() and torch.isnan(v[4, 32:]).all()
    assert not torch.isnan(v[3, 32:]).any() and not torch.isnan(v[4, :32]).any()


def test_quantize_strides_shapes_and_alignment():
    base = torch.randn(40, 320, generator=gen(), device="cuda")
    for x in (base[0, :64], base[:, :96], base[::2, 64:256], base.t()[:, :32], base[:, 2:66], base[3:4, :64],
              base.view(5, 8, 320)[:, 2:5, :160], base.bfloat16()[:, 8:104]):
        q = mx.quantize(x)
        assert q.shape == tuple(x.shape)
        check_quantized(mx.MxTensor(q.codes.reshape(-1, q.codes.shape[-1]),
                                    q.scales.reshape(-1, q.scales.shape[-1])),
                        x.reshape(-1, x.shape[-1]))
    out = mx.MxTensor(torch.zeros(40, 48, dtype=torch.uint8, device="cuda"),
                      torch.zeros(40, 3, dtype=torch.uint8, device="cuda"))
    assert mx.quantize(base[:, :96], out=out) is not None
    check_quantized(out, base[:, :96])
    q = mx.quantize(base[:, :96])
    tail = mx.MxTensor(q.codes[7:], q.scales[7:])          # scales at an odd address
    assert torch.equal(mx.dequantize(tail), mx.dequantize(q)[7:])
    empty = mx.quantize(base[:0, :64])
    assert empty.codes.shape == (0, 32) and mx.dequantize(empty).shape == (0, 64)


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat_interleave(16).view(256, 16)
    codes[:, :] = torch.arange(16, dtype=torch.uint8) * 17       # all codes in every row
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1)
    q = mx.MxTensor(codes.cuda(), scales.cuda())
    ref = R.values(codes.numpy(), scales.numpy())
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref.astype(np.float32))           # past fp32: infinity
    got = mx.dequantize(q, torch.float32).cpu()
    assert torch.equal(got.nan_to_num(1.25), want.nan_to_num(1.25)) or torch.equal(
        got[:255], want[:255]) and torch.isnan(got[255]).all()


# ------------------------------------------------------------------- product
def make(rows, K, N, E, seed, spread=0.0):
    """Quantised inputs with scales that differ from block to block."""
    def q(*shape):
        v = torch.randn(*shape, generator=gen(seed + len(shape)), device="cuda")
        f = torch.exp(spread * torch.randn(*shape[:-1], shape[-1] // 32, 1, generator=gen(seed),
                                           device="cuda"))
        return mx.quantize((v.unflatten(-1, (-1, 32)) * f).flatten(-2))
    return q(rows, K), (q(E, N, K) if E else q(N, K))


def ref_values(q):
    return torch.from_numpy(R.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()))


def check_matmul(out, a, w, offsets, silu, before=None):
    av, wv = ref_values(a), ref_values(w)
    if offsets is None:
        offsets, wv = [0, av.shape[0]], wv[None]
    want, bound = R.matmul(av, wv, offsets, silu, EPS[out.dtype])
    got = out.double().cpu()
    used = ~torch.isnan(want)
    worst = ((got - want).abs() / bound)[used]
    assert not worst.numel() or worst.max() <= 1, float(worst.max())
    if before is not None:                     # rows of no expert are left as they were
        assert torch.equal(got[~used], before.double().cpu()[~used])


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,N", [(1, 128, 32), (2, 256, 64), (17, 384, 160), (33, 2048, 288),
                                      (128, 640, 512), (129, 1536, 96), (300, 128, 1056),
                                      (1000, 896, 416)])
def test_dense(rows, K, N, dtype, silu):
    a, w = make(rows, K, N, 0, rows + K + N, 1.0)
    check_matmul(mx.matmul(a, w, silu_mul=silu, dtype=DT[dtype]), a, w, None, silu)


def test_dense_narrow():
    """N = 16, one weight tile with few rows; N = 16 more than a tile."""
    for N in (16, 144):
        a, w = make(70, 256, N, 0, N)
        check_matmul(mx.matmul(a, w), a, w, None, False)


GROUPS = {
    "uneven": [0, 3, 3, 150, 151, 400, 400],
    "empty": [0, 0, 0, 0],
    "last": [0, 0, 0, 0, 77],
    "first": [0, 65, 65, 65],
    "ones": list(range(20)),
    "gap": [10, 20, 20, 200],                  # rows before the first and behind the last
    "many": [min(5 * i, 700) for i in range(129)],
    "large": [0, 1, 1500, 1516],
}


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_grouped(name, silu):
    offs = GROUPS[name]
    E, rows = len(offs) - 1, max(offs[-1] + (23 if name in ("gap", "empty") else 0), 1)
    a, w = make(rows, 384, 224, E, len(offs), 0.5)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    before = torch.randn(rows, 112 if silu else 224, device="cuda").bfloat16()
    out = before.clone()
    assert mx.matmul(a, w, off, silu_mul=silu, out=out) is out
    check_matmul(out, a, w, offs, silu, before)
    again = mx.matmul(a, w, off, silu_mul=silu, out=before.clone())
    assert torch.equal(out, again)


# Large enough for tiles on CTA pairs (over 48 rows per expert, and tiles for most
# of the GPU).
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,N", [(1500, 512, 2304), (1003, 640, 2976), (577, 128, 6176),
                                      (193, 1024, 6304)])
def test_dense_on_pairs(rows, K, N, dtype, silu):
    a, w = make(rows, K, N, 0, rows + K + N, 1.0)
    check_matmul(mx.matmul(a, w, silu_mul=silu, dtype=DT[dtype]), a, w, None, silu)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [384, 1024])
def test_grouped_on_pairs(K, silu):
    """40 experts with all kinds of row counts, rows before the first and behind
    the last left alone; twice the same bits."""
    counts = [0, 1, 15, 16, 17, 32, 33, 191, 192, 193, 0, 0, 383, 384, 385, 700, 96, 97, 31, 2] * 2
    offs = [7]
    for c in counts:
        offs.append(offs[-1] + c)
    rows, E = offs[-1] + 29, len(counts)
    a, w = make(rows, K, 352, E, K, 0.5)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    before = torch.randn(rows, 176 if silu else 352, device="cuda").bfloat16()
    out = mx.matmul(a, w, off, silu_mul=silu, out=before.clone())
    check_matmul(out, a, w, offs, silu, before)
    assert torch.equal(out, mx.matmul(a, w, off, silu_mul=silu, out=before.clone()))
    assert mx.status() == 0


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("mean", [4, 30, 60])
def test_256_experts(mean, silu):
    """The most experts there may be, for every tile size."""
    g = torch.Generator().manual_seed(mean)
    counts = torch.randint(0, 2 * mean + 1, (256,), generator=g)
    counts[5] += 256 * mean - int(counts.sum()) if int(counts.sum()) < 256 * mean else 0
    offs = [0] + counts.cumsum(0).tolist()
    a, w = make(offs[-1], 640, 64, 256, mean, 0.5)
    out = mx.matmul(a, w, torch.tensor(offs, dtype=torch.int32, device="cuda"), silu_mul=silu)
    check_matmul(out, a, w, offs, silu)


def test_pairs_offsets_and_bad_blocks():
    a, w = make(6000, 128, 64, 60, 2)
    for offs in ([6000 - 100 * i for i in range(61)], [0] + [6000, 0] * 30,
                 [2 ** 31 - 1, -2 ** 31] * 30 + [50], [5900] + [10 ** 6] * 60):
        guard = torch.zeros(8000, 64, device="cuda", dtype=torch.bfloat16)
        mx.matmul(a, w, torch.tensor(offs, dtype=torch.int32, device="cuda"), out=guard[1000:7000])
        torch.cuda.synchronize()
        assert not guard[:1000].any() and not guard[7000:].any()
    assert mx.status() == 0
    a, w = make(1500, 512, 2304, 0, 3)
    a.scales[7, 2] = 255
    w.scales[1300, 0] = 255
    nan = torch.isnan(mx.matmul(a, w))
    want = torch.zeros_like(nan)
    want[7], want[:, 1300] = True, True
    assert torch.equal(nan, want)


def test_scales_off_16_bytes():
    """Scale arrays that TMA cannot address (their start, not their pitch)."""
    a, w = make(1500, 512, 2304, 0, 9, 1.0)
    def off(t):
        buf = torch.empty(t.numel() + 16, dtype=torch.uint8, device="cuda")
        v = buf[4:4 + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    b, v = mx.MxTensor(a.codes, off(a.scales)), mx.MxTensor(w.codes, off(w.scales))
    for x, y in ((b, v), (a, v), (b, w)):
        assert torch.equal(mx.matmul(x, y), mx.matmul(a, w))
        few = mx.MxTensor(x.codes[:9], x.scales[:9])
        assert torch.equal(mx.matmul(few, y), mx.matmul(mx.MxTensor(a.codes[:9], a.scales[:9]), w))


def test_empty_batch_and_shapes():
    a, w = make(4, 128, 64, 3, 1)
    none = mx.MxTensor(a.codes[:0], a.scales[:0])
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert mx.matmul(none, w, off).shape == (0, 64)
    assert mx.matmul(none, w, off, silu_mul=True).shape == (0, 32)


def test_offsets_out_of_order_stay_inside():
    """Offsets that descend, or leave [0, rows], give unspecified rows but write
    nothing outside out."""
    a, w = make(50, 128, 64, 4, 2)
    for offs in ([0, 40, 10, 60, 90], [-7, 5, 200, 3, 50], [50, 40, 30, 20, 10],
                 [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0, 50]):
        guard = torch.zeros(250, 64, device="cuda", dtype=torch.bfloat16)
        mx.matmul(a, w, torch.tensor(offs, dtype=torch.int32, device="cuda"), out=guard[100:150])
        torch.cuda.synchronize()
        assert not guard[:100].any() and not guard[150:].any()


def test_bad_block_stays_in_its_row():
    """A NaN scale of a row reaches that row alone, one of a weight row that
    output column alone."""
    a, w = make(40, 256, 64, 0, 3)
    a.scales[7, 2] = 255
    out = mx.matmul(a, w)
    assert torch.isnan(out[7]).all() and not torch.isnan(out[:7]).any()
    assert not torch.isnan(out[8:]).any()
    a, w = make(40, 256, 64, 0, 3)
    w.scales[9, 0] = 255
    out = mx.matmul(a, w)
    assert torch.isnan(out[:, 9]).all() and not torch.isnan(out[:, :9]).any()
    assert not torch.isnan(out[:, 10:]).any()


def test_scales_far_apart():
    """Scales near both ends of what fp32 sums can hold."""
    a, w = make(8, 256, 64, 0, 4)
    a.scales.fill_(40)
    w.scales.fill_(200)
    check_matmul(mx.matmul(a, w, dtype=torch.float32), a, w, None, False)


def test_refusals():
    a, w = make(4, 128, 64, 2, 1)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mx.matmul(a, w)                                    # experts without offsets
    with pytest.raises(ValueError):
        mx.matmul(a, w, off.long())
    with pytest.raises(ValueError):
        mx.matmul(a, w, off[:2])
    with pytest.raises(ValueError):
        mx.matmul(a, w, off, out=torch.empty(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        mx.matmul(mx.MxTensor(a.codes[:, :32], a.scales[:, :2]), w, off)
    b, v = make(4, 96, 64, 0, 1)
    with pytest.raises(MoeError) as e:
        mx.matmul(b, v)                                    # K % 128
    assert e.value.code == -2
    with pytest.raises(ValueError):
        mx.quantize(torch.zeros(4, 40, device="cuda"))


# ----------------------------------------------------------- streams, graphs
def test_other_stream_and_graph():
    """On a stream that is not the current one, and captured: replays read the
    inputs' new contents."""
    a, w = make(64, 256, 128, 3, 5)
    off = torch.tensor([0, 10, 40, 64], dtype=torch.int32, device="cuda")
    x = torch.randn(64, 256, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = mx.quantize(x, stream=s)
    y = mx.matmul(q, w, off, stream=s)
    s.synchronize()
    check_quantized(q, x)
    check_matmul(y, q, w, off.tolist(), False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq = mx.quantize(x)
        gv = mx.dequantize(gq)
        gy = mx.matmul(gq, w, off, silu_mul=True)
    for seed in (1, 2):
        x.copy_(torch.randn(64, 256, generator=gen(seed), device="cuda"))
        off.copy_(torch.tensor([0, 0, 5 * seed, 60 + seed], dtype=torch.int32))
        gy.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_quantized(gq, x)
        assert torch.equal(gv, mx.dequantize(gq))
        check_matmul(gy, gq, w, off.tolist(), True, torch.zeros_like(gy))


@pytest.mark.parametrize("rows,N", [(700, 256), (5000, 2048)])
def test_two_streams_at_once(rows, N):
    a, w = make(rows, 512, N, 4, 6)
    offs = [[0, 100, 300, 301, rows], [0, 0, 0, 690, rows]]
    off = [torch.tensor(o, dtype=torch.int32, device="cuda") for o in offs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s, o in zip(streams, off):
            outs.append(mx.matmul(a, w, o, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, outs[i % 2])
    for i in (0, 1):
        check_matmul(outs[i], a, w, offs[i], False)
