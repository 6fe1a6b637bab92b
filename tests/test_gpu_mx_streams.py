"""Inputs and outputs of the MXFP4 calls that are dropped while a call on another
stream has yet to read or write them: their memory must not be handed out until
then. The other stream is held up by a sleep, and the memory is asked for again
and overwritten at once."""
import pytest
import torch

from sigmoid_bias_top_b200 import mx

pytestmark = pytest.mark.gpu
SLEEP = 100_000_000        # cycles: 50 ms and more
ROWS, K, N = 4096, 2048, 256


def held_up():
    s = torch.cuda.Stream()
    for dt in (torch.bfloat16, torch.uint8, torch.int32):    # a kernel's first launch would wait
        torch.empty(8, dtype=dt, device="cuda").fill_(99)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    return s


def overwrite(*like):
    """New tensors of the dropped ones' sizes; kept until the caller is done."""
    new = [torch.empty_like(t, device="cuda") for t in like]
    for t in new:
        t.fill_(99)
    return new


def data(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(ROWS, K, generator=g, device="cuda").bfloat16()


def test_quantize_input_dropped():
    for _ in range(2):                 # the process's first calls may take longer than the sleep
        want, meta = mx.quantize(data(1)), torch.empty(ROWS, K, dtype=torch.bfloat16, device="meta")
        torch.cuda.empty_cache()
        x = data(1)
        s = held_up()
        q = mx.quantize(x, stream=s)
        del x
        keep = overwrite(meta, meta)
        s.synchronize()
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
        assert len(keep) == 2


def test_dequantize_input_dropped():
    q = mx.quantize(data(2))
    want = mx.dequantize(q)
    metas = [t.to("meta") for t in q]
    torch.cuda.empty_cache()
    s = held_up()
    y = mx.dequantize(q, stream=s)
    del q
    keep = overwrite(*metas, *metas)
    s.synchronize()
    assert torch.equal(y, want) and len(keep) == 4


@pytest.mark.parametrize("grouped", [False, True])
def test_matmul_inputs_dropped(grouped):
    def make():
        w = mx.quantize(data(4)[:2 * N].view(2, N, K) if grouped else data(4)[:N].contiguous())
        off = torch.tensor([0, 1000, ROWS], dtype=torch.int32, device="cuda") if grouped else None
        return mx.quantize(data(3)), w, off
    a, w, off = make()
    want = mx.matmul(a, w, off)
    metas = [t.to("meta") for t in (*a, *w) + ((off,) if grouped else ())]
    torch.cuda.empty_cache()
    s = held_up()
    y = mx.matmul(a, w, off, stream=s)
    del a, w, off
    keep = overwrite(*metas, *metas)
    s.synchronize()
    assert torch.equal(y, want) and keep


def test_outputs_dropped():
    """An output given and dropped: what is made of its memory next stays as it is."""
    q = mx.quantize(data(5))
    out = torch.empty(ROWS, K, dtype=torch.bfloat16, device="cuda")
    meta = out.to("meta")
    s = held_up()
    mx.dequantize(q, out=out, stream=s)
    del out
    keep = overwrite(meta, meta)
    torch.cuda.current_stream().synchronize()
    s.synchronize()
    assert all((t == 99).all() for t in keep)


def test_on_a_forked_stream_of_a_capture():
    """quantize and matmul on a stream that joins the capture; their tensors may go
    once it is captured, and the next eager calls are not disturbed."""
    x, w = data(6), mx.quantize(data(7)[:N].contiguous())
    want = mx.matmul(mx.quantize(x), w)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        s.wait_stream(main)
        q = mx.quantize(x, stream=s)
        y = mx.matmul(q, w, stream=s)
        del q
        main.wait_stream(s)
    for seed in (6, 8):
        x.copy_(data(seed))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) == (seed == 6)
        assert torch.equal(y, mx.matmul(mx.quantize(x), w))
    del g, y
    assert torch.equal(mx.matmul(mx.quantize(data(6)), w), want) and mx.status() == 0
