"""Other Python threads while an operator allocates and launches."""
import threading
import time

import pytest
import torch

import ring_all_reduce_allreduce_amd as rs

pytestmark = pytest.mark.gpu


def test_other_threads_run_during_a_call():
    """A list of a million entries takes 3031 launches, some ten milliseconds
    in the library. A thread that wakes up every half one runs meanwhile; it
    could run once or twice, around the call, if the call kept the
    interpreter to itself."""
    g = torch.full((1024,), 0.5, device="cuda")
    grads = (g,) * 1_000_000
    rs.grad_norm(grads[:1000])
    ticks, done = [], threading.Event()

    def tick():
        while not done.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.0005)

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        time.sleep(0.01)
        begin = time.perf_counter()
        norm = rs.grad_norm(grads)
        end = time.perf_counter()
    finally:
        done.set()
        thread.join()
    assert abs(float(norm) - 16_000.0) < 0.01  # 0.5 sqrt(1024 * 10^6)
    assert sum(begin < t < end for t in ticks) >= 5


def test_two_threads_on_two_streams():
    """Calls from two threads, each on a stream of its own, give what one
    thread's calls give."""
    x = [torch.randn(700, 1000, device="cuda").bfloat16() for _ in range(2)]
    w = torch.ones(1000, device="cuda", dtype=torch.bfloat16)
    lists = [[torch.randn(n, device="cuda") for n in (100_003, 17, 5_000)] for _ in range(2)]
    want = [(rs.rms_norm(a, w), rs.rms_norm_backward(a, a, w), rs.grad_norm(g)) for a, g in zip(x, lists)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                n, b, norm = rs.rms_norm(x[i], w), rs.rms_norm_backward(x[i], x[i], w), rs.grad_norm(lists[i])
                stream.synchronize()
                if not (torch.equal(n.out, want[i][0].out) and torch.equal(b.grad_in, want[i][1].grad_in)
                        and torch.equal(b.grad_weight, want[i][1].grad_weight) and torch.equal(norm, want[i][2])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
