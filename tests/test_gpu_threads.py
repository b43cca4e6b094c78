"""Calls of the native tensor binding beside other Python threads."""
import threading
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_448_b200 as pk
from gpu_helpers import i32

pytestmark = pytest.mark.gpu


def calls():
    planes = pk.mxfp4_cache(8, 1, 16, 64)
    rows = [torch.randn(4, 1, 64, device="cuda").half() for _ in range(2)]
    q, out = (torch.zeros(2, 1, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    slots, table, ctx, cu = i32(np.arange(4)), i32([[0], [1]]), i32([4, 3]), i32([0, 1, 2])
    dws = pk.decode_workspace(2, 1, 1, 64, 16, 16, cache_dtype=pk.PA_MXFP4)
    cws = pk.chunked_prefill_workspace(2, 2, 1, 1, 64, 1, 16, pk.PA_MXFP4)
    pool = pk.CachePool(planes, 16)
    nt, nc = i32([[0]]), i32([0])
    zero, seven, moves = i32([0]), i32([7]), i32([[3, 2]])
    return {
        "write": lambda: pk.reshape_and_cache_mxfp4(*rows, *planes, slots),
        "read": lambda: pk.gather_cache_mxfp4(*rows, *planes, slots),
        "decode": lambda: pk.decode_mxfp4(out, q, *planes, table, ctx, 16, 0.1, workspace=dws),
        "chunk": lambda: pk.chunked_prefill_mxfp4(out, q, cu, 1, *planes, table, ctx, 16, 0.1,
                                                  workspace=cws),
        "fork": lambda: pool.fork(table, ctx, zero, seven, nt, nc),
        "compact": lambda: pool.compact(moves)}


@pytest.mark.parametrize("name", ["write", "read", "decode", "chunk", "fork", "compact"])
def test_other_threads_run_while_a_call_waits_for_the_queue(name):
    """A kernel of about half a second, then more calls than the GPU's queue takes: the call that
    waits for room does not hold up the other Python threads."""
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def tick():
        last = time.monotonic()
        while not stop.is_set():
            time.sleep(0.005)
            now = time.monotonic()
            gaps.append(now - last)
            last = now
    thread = threading.Thread(target=tick)
    thread.start()
    try:
        torch.cuda._sleep(1_000_000_000)
        longest = 0.0
        for _ in range(3000):
            t = time.monotonic()
            call()
            longest = max(longest, time.monotonic() - t)
    finally:
        stop.set()
        thread.join()
        torch.cuda.synchronize()
    assert longest > 0.2, "no call waited: the queue did not fill"
    assert max(gaps) < longest / 2, f"a thread stood still for {max(gaps):.2f} s"
