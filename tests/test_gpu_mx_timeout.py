"""Waits of the MXFP4 product that run out: barriers of one kind wait for an
arrival that nothing makes, so that each role in turn is the one to give up, on
single CTAs and on pairs. The call ends, the status tells of it once, and the
next product is right (its TMEM, barriers and shared memory are its own)."""
import pytest
import torch

from sigmoid_bias_top_b200 import MOE_BF16, mx

pytestmark = pytest.mark.gpu
TIMEOUT = -7
FULL_A, SCALED_A, EMPTY_A, FULL_B, SCALED_B, EMPTY_B, T_FULL, T_EMPTY, DEALT, TAKEN = range(1, 11)


def make(rows, K, N, E):
    g = torch.Generator(device="cuda").manual_seed(rows + E)
    a = mx.quantize(torch.randn(rows, K, generator=g, device="cuda").bfloat16())
    w = mx.MxTensor(*(torch.randint(lo, hi, (E, N, K // d), generator=g, device="cuda",
                                    dtype=torch.uint8) for d, lo, hi in ((2, 0, 256), (32, 120, 124))))
    off = torch.linspace(0, rows, E + 1, device="cuda").round().int()
    return a, w, off


def run(a, w, off, withheld, timeout_us=3000, silu=False):
    rows, K, (E, N) = a.codes.shape[0], a.shape[1], w.codes.shape[:2]
    out = torch.empty(rows, N // 2 if silu else N, dtype=torch.bfloat16, device="cuda")
    assert mx.lib().moe_mx_selftest_timeout(
        a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
        off.data_ptr(), rows, K, E, N, int(silu), out.data_ptr(), MOE_BF16, timeout_us, withheld,
        torch.cuda.current_stream().cuda_stream) == 0
    return out


def check(case, kinds, silu=False):
    a, w, off = make(*case)
    want = mx.matmul(a, w, off, silu_mul=silu)
    assert mx.status() == 0
    for kind in kinds:
        run(a, w, off, kind, silu=silu)
        assert mx.status() == TIMEOUT, kind
        assert mx.status() == 0, kind
        assert torch.equal(mx.matmul(a, w, off, silu_mul=silu), want), kind
        assert mx.status() == 0, kind
    # the same call with nothing withheld, and with a limit that it keeps
    assert torch.equal(run(a, w, off, 0, 1000000, silu), want) and mx.status() == 0


def test_single_cta_first_items():
    check((17, 256, 128, 1), [FULL_B, T_FULL, DEALT])


def test_single_ctas():
    """Over 32 items a CTA, tiles of 32 rows, scales by TMA."""
    check((256, 512, 2432, 256), [FULL_B, SCALED_B, EMPTY_B, T_FULL, T_EMPTY, DEALT, TAKEN])


@pytest.mark.parametrize("silu", [False, True])
def test_single_ctas_of_48_rows(silu):
    """Scales loaded by the warps."""
    check((1600, 1152, 2560, 40), [FULL_B, EMPTY_B, T_FULL, T_EMPTY, DEALT], silu)


def test_pairs():
    """Over 32 items a pair, a run's weights shared, scales by TMA."""
    check((8000, 512, 8192, 40), [FULL_A, SCALED_A, EMPTY_A, FULL_B, SCALED_B, EMPTY_B, T_FULL, T_EMPTY,
                                  DEALT, TAKEN])


@pytest.mark.parametrize("silu", [False, True])
def test_pairs_of_long_rows(silu):
    """Weights loaded for every item, scales loaded by the warps."""
    check((4000, 2688, 2048, 20), [FULL_A, EMPTY_A, FULL_B, EMPTY_B, T_FULL, T_EMPTY, DEALT], silu)


def test_a_layer_reports_its_own():
    """A time-out of a call without a context is not a layer's."""
    from sigmoid_bias_top_b200 import MoeLayer, workloads as W
    w = W.DECODE.scaled(n_tokens=20, d=256, n_experts=16, top_k=4, d_ff=128)
    m = MoeLayer(mx.quantize_experts(W.make_layer(w, 0, "cuda")), 4, w.eps, max_tokens=20)
    x = W.make_x(w, "cuda")
    want = m(x)
    a, wt, off = make(17, 256, 128, 1)
    run(a, wt, off, FULL_B)
    assert torch.equal(m(x), want) and m.status() == 0
    assert mx.status() == TIMEOUT and mx.status() == 0
    m.close()


def test_every_thread_is_told():
    """One thread's reading does not take a time-out from another's."""
    from concurrent.futures import ThreadPoolExecutor
    a, w, off = make(17, 256, 128, 1)
    with ThreadPoolExecutor(1) as other:
        def status():
            return other.submit(mx.status, "cuda:0").result()
        status(), mx.status()
        run(a, w, off, FULL_B)
        assert status() == TIMEOUT and mx.status() == TIMEOUT
        assert status() == 0 and mx.status() == 0
        run(a, w, off, FULL_B)
        assert mx.status() == TIMEOUT and status() == TIMEOUT
        assert mx.status() == 0 and status() == 0
