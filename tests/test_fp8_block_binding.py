"""The Python binding beside other threads and streams."""
import threading
import time

import numpy as np
import pytest
import torch

from test_fp8_block_long import _bf16, _dev, _i32, _pools, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa


def _decode_args(n=64):
    rng = np.random.default_rng(1)
    pools = _dev(*_pools(rng, 8, 16, 1))
    q = _bf16(rng, (1, 4, 128)).cuda()
    ws = pa.new_decode_fp8_block_workspace(1, 4, 1, 128, 16, n)
    return (q, *pools, _i32(np.arange(4)[None]), _i32([n]), n, 0.1, ws)


@pytest.mark.gpu
def test_a_full_launch_queue_stops_no_other_thread():
    """Calls that wait for room in the launch queue, behind half a second of other work, let other Python threads run."""
    args, out = _decode_args(), torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_fp8_block(*args, out=out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    cycles = int(0.5 * 1e3 * torch.cuda.get_device_properties(0).clock_rate) if hasattr(
        torch.cuda.get_device_properties(0), "clock_rate") else int(1e9)
    times = {}

    def calls():
        with torch.cuda.stream(s):
            torch.cuda._sleep(cycles)
            times["start"] = time.perf_counter()
            for _ in range(4000):
                pa.pa_decode_fp8_block(*args, out=out, stream=s)
            times["end"] = time.perf_counter()

    t = threading.Thread(target=calls)
    gap, last = 0.0, time.perf_counter()
    t.start()
    while t.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    t.join()
    torch.cuda.synchronize()
    assert times["end"] - times["start"] > 0.2, "the queue took every call at once: the test shows nothing"
    assert gap < 0.25, f"another thread stood still for {gap:.2f} s"


def _calls():
    """Calls that take a stream and allocate their output, by name; their inputs are ready and kept."""
    args = _decode_args()
    q, *pools, bt, ctx, n, scale, _ = args
    cu, start, seq, pos = _i32([0, 1]), _i32([n - 1]), _i32([0]), _i32(range(4))
    first = _i32([0] * 4)
    kb, vb = (torch.ones(8, 16, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = pa.new_decode_workspace(1, 4, 1, 128, 16, n)
    return {
        "decode": lambda stream: pa.pa_decode_fp8_block(*args, stream=stream),
        "prefill": lambda stream: pa.pa_prefill_chunk_fp8_block(q, cu, start, seq, 1, *pools, bt, ctx, n, scale,
                                                                stream=stream),
        "read": lambda stream: pa.pa_read_kv_paged_fp8_block(*pools, bt, first, pos, stream=stream)[0],
        "bf16 decode": lambda stream: pa.pa_decode(q, kb, vb, bt, ctx, n, scale, ws, stream=stream),
        "bf16 prefill": lambda stream: pa.pa_prefill_chunk(q, cu, start, seq, 1, kb, vb, bt, ctx, scale, stream=stream),
        "slots": lambda stream: pa.pa_slot_mapping(bt, first, pos, 16, 8, stream=stream),
        "tables": lambda stream: pa.pa_map_to_kernel_blocks(bt, 2, stream=stream),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode", "prefill", "read", "bf16 decode", "bf16 prefill", "slots",
                                  "tables"])
def test_outputs_that_are_not_given_belong_to_the_given_stream(name):
    """Memory that other streams may still use is not handed out: of what the current stream freed, to a call on another;
    of a dropped output, to the current stream; of an output in use by the current stream, to the given one."""
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    cycles = int(2e8)  # a tenth of a second

    held = torch.empty_like(want)
    freed = held.data_ptr()
    torch.cuda._sleep(cycles)
    held.fill_(3)  # still to come when the call below runs
    del held
    got = call(other)
    assert got.data_ptr() != freed
    torch.cuda.synchronize()
    assert torch.equal(got, want)

    with torch.cuda.stream(other):
        torch.cuda._sleep(cycles)
    got = call(other)
    dropped = got.data_ptr()
    del got
    again = torch.empty_like(want)
    assert again.data_ptr() != dropped
    torch.cuda.synchronize()

    got = call(other)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(cycles)
    copy, used = got.clone(), got.data_ptr()
    del got
    with torch.cuda.stream(other):
        more = [torch.empty_like(want) for _ in range(4)]
    assert all(m.data_ptr() != used for m in more)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    for handle in (other.cuda_stream, torch.cuda.default_stream().cuda_stream):  # a stream given as a number
        got = call(handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
