"""What fa_sync_status costs: one launch, one copy and one wait, whatever the
number of translation units that keep a status word."""
from __future__ import annotations

import statistics
import threading
import time

import pytest
import torch

from exact_attention_10_gb300 import fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()


def _median_us(f, n=300):
    times = []
    for i in range(n + 20):
        t = time.perf_counter()
        f()
        times.append(time.perf_counter() - t)
    return statistics.median(times[20:]) * 1e6


def test_status_costs_one_launch_copy_and_wait():
    """Less than one and a half of torch's reads of a fresh result (a launch, a copy
    and a wait); a launch, copy and wait for each of seven words takes 3.4."""
    x = torch.zeros(1, device="cuda")
    st = torch.cuda.current_stream().cuda_stream

    def one():
        torch.cuda.synchronize()
        return x.add_(1).item()

    # (in turn, so that both see the same machine)
    ratios = []
    for _ in range(5):
        base = _median_us(one)
        ratios.append(_median_us(lambda: fa.sync_status(st)) / base)
    print("status / (launch, copy, wait):", ratios)
    assert statistics.median(ratios) < 1.5, ratios


def test_status_from_many_threads():
    """Calls on streams of their own from eight threads at a time, beside work."""
    got, q = [], torch.randn((1, 2, 300, 64), device="cuda").bfloat16()
    want = fa.forward(q, q, q, causal=True)[0]
    torch.cuda.synchronize()

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                o, _ = fa.forward(q, q, q, causal=True)
                got.append((fa.sync_status(s.cuda_stream), torch.equal(o, want)))

    threads = [threading.Thread(target=work) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 400 and all(rc == 0 and same for rc, same in got)
