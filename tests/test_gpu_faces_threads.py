"""The compiled faces let other Python threads run while a call waits for room in the GPU's queue."""
import threading
import time

import pytest

pytestmark = pytest.mark.gpu


def _calls():
    import torch
    from block_diffusion_speculative_hidden_gb300 import (Fp4, PagePool, copy_pages, dequantize_fp4, fork_pages, gemm_fp4,
                                                          quantize_fp4, truncate_pages, verify_tokens)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    t = quantize_fp4(x)
    out, y = torch.empty(4, 4, device="cuda"), torch.empty(4, 64, device="cuda")
    k = torch.zeros(1, 8, 1, 16, 32, device="cuda")
    pool = PagePool(k, k.clone(), torch.full((3, 2), -1, **i32), torch.zeros(3, **i32), torch.zeros(8, **i32))
    one, two = torch.zeros(1, **i32), torch.ones(1, **i32)
    p = torch.full((1, 2, 8), 0.125, device="cuda")
    tok, ua, us = torch.zeros(1, 1, **i32), torch.zeros(1, 1, device="cuda"), torch.zeros(1, device="cuda")
    a, n = torch.zeros(1, 2, **i32), torch.zeros(1, **i32)
    ws = torch.empty(pool.workspace(), dtype=torch.uint8, device="cuda")
    return {"quantise": lambda: quantize_fp4(x, out=t), "take back": lambda: dequantize_fp4(t, out=y),
            "product": lambda: gemm_fp4(t, t, out=out), "verify": lambda: verify_tokens(tok, p, ua, us, out=a, n_out=n),
            "fork": lambda: fork_pages(pool, one, two, workspace=ws), "cut": lambda: truncate_pages(pool, one, seq=one),
            "copy": lambda: copy_pages(pool, one, two)}


@pytest.mark.parametrize("name", ["quantise", "take back", "product", "verify", "fork", "cut", "copy"])
def test_other_threads_run_while_a_call_waits(name):
    import torch
    call = _calls()[name]
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)
    other = threading.Thread(target=tick)
    other.start()
    try:
        time.sleep(0.05)
        torch.cuda._sleep(2_000_000_000)             # a second of the GPU
        t0, longest = time.perf_counter(), 0.0
        for _ in range(6000):                        # far more than the queue has room for
            t = time.perf_counter()
            call()
            longest = max(longest, time.perf_counter() - t)
        t1 = time.perf_counter()
    finally:
        stop.set()
        other.join()
    torch.cuda.synchronize()
    if longest < 0.3:
        pytest.skip("no call waited")
    seen = [t for t in ticks if t0 <= t <= t1]
    gap = max(b - a for a, b in zip([t0, *seen], [*seen, t1]))
    assert gap < longest / 2, (gap, longest)
