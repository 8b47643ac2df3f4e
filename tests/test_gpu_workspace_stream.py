"""A decode on another stream than the current one: its workspace is not handed on while the call still runs."""
import pytest
import torch

import q8_window_ref as R
from test_gpu_q8_window import Device, Q  # noqa: F401

pytestmark = pytest.mark.gpu

CALLS = [("q8", 0), ("q8", 700), ("bf16", 700), ("bf16", 0)]       # 8-bit, windowed, and the call with neither


def arguments(dev, c):
    return (*dev.in_, dev.kv, dev.ak, dev.lens, dev.table, c.page, c.max_pages, c.G, c.scale, R.EPS, dev.o, dev.lse)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("cache,window", CALLS)
def test_decode_on_another_stream(Q, cache, window, raw):  # noqa: F811
    c = R.Case([1500, 700], cache=cache, window=window)
    dev = Device(Q, c, num_splits=3)
    need = dev.call.workspace.numel()
    dev.call()
    torch.cuda.synchronize()
    want = dev.o.clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        dev.o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)
        Q.decode(*arguments(dev, c), num_splits=3, kv_scale=dev.scale, window=window,
                 stream=side.cuda_stream if raw else side)
        # the current stream goes on at once: whatever it allocates is its own
        own = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert all(bool((x == 7).all()) for x in own)
        assert torch.equal(dev.o, want)
    assert Q.get_device_status() == 0


@pytest.mark.parametrize("cache,window", CALLS)
def test_prepared_call_dropped_on_another_stream(Q, cache, window):  # noqa: F811
    c = R.Case([1500, 700], cache=cache, window=window)
    dev = Device(Q, c, num_splits=3)
    need = dev.call.workspace.numel()
    dev.call()
    torch.cuda.synchronize()
    want = dev.o.clone()
    side = torch.cuda.Stream()
    dev.o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2000000)
    dev.call(side)
    dev.call(side)
    del dev.call
    own = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in own)
    assert torch.equal(dev.o, want)


def test_workspace_made_behind_pending_work(Q):  # noqa: F811
    """The memory of a new workspace may still be in use on the stream it comes from: a call on another stream
    waits for that."""
    c = R.Case([1500, 700], window=700)
    dev = Device(Q, c, num_splits=3)
    need = dev.call.workspace.numel()
    dev.call()
    torch.cuda.synchronize()
    want = dev.o.clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        dev.o.zero_()
        old = torch.empty(need, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(2000000)
        old.fill_(255)
        del old
        call = Q.prepare_decode(*arguments(dev, c), num_splits=3, kv_scale=dev.scale, window=700)
        call(side)
        torch.cuda.synchronize()
        assert torch.equal(dev.o, want)


@pytest.mark.parametrize("cache,window", CALLS)
def test_decode_on_the_default_stream_by_handle(Q, cache, window):  # noqa: F811
    """Handle 0 is the default stream, also where another one is current."""
    c = R.Case([1500, 700], cache=cache, window=window)
    dev = Device(Q, c, num_splits=3)
    need = dev.call.workspace.numel()
    dev.call()
    torch.cuda.synchronize()
    want = dev.o.clone()
    dev.o.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(2000000)                                     # on the default stream
    with torch.cuda.stream(torch.cuda.Stream()):
        Q.decode(*arguments(dev, c), num_splits=3, kv_scale=dev.scale, window=window, stream=0)
        own = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in own)
    assert torch.equal(dev.o, want)
    assert Q._stream_object(0) == torch.cuda.default_stream()
