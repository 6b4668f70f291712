"""The native binding of the mixer operators beside other Python threads."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_other_threads_run_while_a_call_waits():
    """A launch waits where the stream's queue is full (it holds about a
    thousand); Python's lock is free meanwhile.  The longest pause of a thread
    that does little but look at the clock stays well below the time for which
    the queue is held up."""
    import kalman_linear_attention_b200 as kla
    f, x, h = (torch.rand(2, 3, 8, device=DEV) for _ in range(3))
    kla.gated_scan_step(f, x, h)
    torch.cuda.synchronize()
    stop, pauses = threading.Event(), []

    def look():
        last, longest = time.perf_counter(), 0.0
        while not stop.is_set():
            now = time.perf_counter()
            longest, last = max(longest, now - last), now
            time.sleep(1e-4)
        pauses.append(longest)

    clock = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    thread = threading.Thread(target=look)
    thread.start()
    clock[0].record()
    torch.cuda._sleep(int(1.5e9))  # cycles: about 0.8 s
    clock[1].record()
    start = time.perf_counter()
    for _ in range(4000):
        kla.gated_scan_step(f, x, h)
    waited = time.perf_counter() - start
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    held_up = clock[0].elapsed_time(clock[1]) / 1e3
    assert waited > held_up / 2, "the queue was not full"
    assert pauses[0] < held_up / 4, (pauses, held_up, waited)
