"""slim_async_status: a bounded wait of the grouped product made to run out (a limit of no polls on the epilogue's wait,
for tests only) ends the call within its limits, is reported once, and leaves the device usable."""
import time

import pytest
import torch

import grouped_util as U
from post_weight_quantization_hessian_b200 import slim

pytestmark = pytest.mark.gpu

ETIMEOUT, EPILOGUE_WAIT = 4, 11


def setup(R, n=2048, m=1000, group=64, dtype=torch.bfloat16):
    layer = U.random_layers(1, m, n, group, 2, R)
    x = torch.randn((R, n), device="cuda").to(dtype)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    return lambda **kw: slim.slim_dequant_grouped_gemm(*layer, group, 2, x, off, **kw)


@pytest.mark.parametrize("R, group, dtype", [(40, 64, torch.bfloat16), (700, 64, torch.bfloat16), (700, 32, torch.float32),
                                             (5000, 128, torch.bfloat16)])
def test_a_wait_that_runs_out(monkeypatch, R, group, dtype):
    call = setup(R, group=group, dtype=dtype)
    want = call()
    slim.slim_async_status()
    monkeypatch.setenv("SLIM_TEST_GROUPED_POLLS", "0")
    t0 = time.monotonic()
    call()
    with pytest.raises(slim.SlimError) as e:
        slim.slim_async_status()
    # the roles notice within polls of 20 us, and copies and products in flight end at once: no wait of 2 s runs out
    assert time.monotonic() - t0 < 1.0
    assert e.value.status == ETIMEOUT and e.value.device_detail == EPILOGUE_WAIT
    slim.slim_async_status()                                  # reported once
    monkeypatch.delenv("SLIM_TEST_GROUPED_POLLS")
    assert torch.equal(call(), want)
    slim.slim_async_status()


def test_failures_of_another_stream_are_kept_for_the_next_query(monkeypatch):
    call, other = setup(300), torch.cuda.Stream()
    want = call()
    slim.slim_async_status()
    monkeypatch.setenv("SLIM_TEST_GROUPED_POLLS", "0")
    call()
    torch.cuda.synchronize()
    with pytest.raises(slim.SlimError):
        slim.slim_async_status(stream=other)                  # the device's status, whichever stream asks
    reported, calls = 0, 20
    for _ in range(calls):                                    # failures of one stream, queries on another
        call(stream=other)
        try:
            slim.slim_async_status()
        except slim.SlimError as e:
            assert e.status == ETIMEOUT
            reported += 1
    other.synchronize()
    try:
        slim.slim_async_status()
    except slim.SlimError:
        reported += 1
    assert 1 <= reported <= calls
    slim.slim_async_status()
    monkeypatch.delenv("SLIM_TEST_GROUPED_POLLS")
    assert torch.equal(call(), want)
    slim.slim_async_status()


def test_captured_call_reports(monkeypatch):
    call = setup(200)
    monkeypatch.setenv("SLIM_TEST_GROUPED_POLLS", "0")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        g.replay()
        with pytest.raises(slim.SlimError):
            slim.slim_async_status()
    slim.slim_async_status()


def test_refused_on_a_stream_that_is_being_captured():
    call = setup(200)
    want = call()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = call()
        with pytest.raises(slim.SlimError) as e:
            slim.slim_async_status()
    assert e.value.status == 1
    g.replay()
    slim.slim_async_status()
    assert torch.equal(got, want)
