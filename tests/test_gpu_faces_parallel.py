"""Calls of several Python threads at once, each on a stream of its own, with outputs that the calls make."""
import threading

import pytest

pytestmark = pytest.mark.gpu


def test_threads_beside_each_other():
    import torch
    from block_diffusion_speculative_hidden_gb300 import (PagePool, dequantize_fp4, fork_pages, gemm_fp4, quantize_fp4,
                                                          reserve_pages, truncate_pages, verify_tokens)
    from fp4_ref import untile
    g = torch.Generator(device="cuda").manual_seed(1)
    w = quantize_fp4(torch.randn(640, 512, generator=g, device="cuda"), "nv", scale=torch.full((1,), 0.01, device="cuda"))
    xs = [torch.randn(17 + 30 * i, 512, generator=g, device="cuda") for i in range(4)]
    p = torch.softmax(torch.randn(9, 4, 3000, generator=g, device="cuda"), -1)
    tok = torch.randint(0, 3000, (9, 3), generator=g, device="cuda").int()
    ua, us = torch.rand(9, 3, generator=g, device="cuda"), torch.rand(9, generator=g, device="cuda")

    def step(i):
        i32 = dict(dtype=torch.int32, device="cuda")
        t = quantize_fp4(xs[i], "nv")
        out, back = gemm_fp4(w, t, dtype=torch.float32), dequantize_fp4(t)
        a, n = verify_tokens(tok, p, (ua + i / 4) % 1, us)
        k = torch.zeros(1, 40, 1, 16, 32, device="cuda")
        pool = PagePool(k, k.clone(), torch.full((6, 4), -1, **i32), torch.zeros(6, **i32), torch.zeros(40, **i32))
        reserve_pages(pool, torch.tensor([20 + i, 7], **i32))
        fork_pages(pool, torch.tensor([0, 1, 0], **i32), torch.tensor([3, 4, 5], **i32))
        truncate_pages(pool, torch.tensor([3 + i], **i32))
        # (the tiles' rows behind the last one are not written)
        scales = untile(t.scales, *xs[i].shape, "nv")
        return [out, back, a, n, w.codes, t.codes, scales, pool.page_table, pool.seq_len, pool.refs]
    want = [[x.clone() for x in step(i)] for i in range(4)]
    torch.cuda.synchronize()
    wrong, rounds = [], 40

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(rounds):
                    for a, b in zip(step(i), want[i]):
                        if not torch.equal(a.nan_to_num(3.0), b.nan_to_num(3.0)):
                            wrong.append((i, a, b))
        except Exception as e:                       # noqa: BLE001 (reported below)
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:2]
