"""The compiled binding beside other threads and streams."""
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
    assert gap < 0.1, f"another thread stood still for {gap:.2f} s"
