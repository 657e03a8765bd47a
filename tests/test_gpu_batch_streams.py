"""The batch operators over two streams that wait for each other, eagerly and recorded: a step whose products run beside
its page calls, over buffers that are written again at once."""
import pytest

pytestmark = pytest.mark.gpu


class Work:
    def __init__(self):
        import torch
        from block_diffusion_speculative_hidden_gb300 import Fp4, PagePool, quantize_fp4, reserve_pages
        g = torch.Generator("cuda").manual_seed(5)
        i32 = dict(dtype=torch.int32, device="cuda")
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.W = quantize_fp4(torch.randn(1500, 512, generator=g, device="cuda") * 0.05, "nv")
        self.x = torch.randn(60, 512, generator=g, device="cuda").bfloat16()
        self.t = Fp4(torch.empty(60, 256, **u8), torch.zeros(4096, **u8), "nv")
        self.logits, self.p = torch.empty(60, 1500, device="cuda"), torch.empty(12, 5, 1500, device="cuda")
        self.tok = torch.randint(0, 1500, (12, 4), generator=g, device="cuda").int()
        self.ua, self.us = torch.rand(12, 4, generator=g, device="cuda"), torch.rand(12, generator=g, device="cuda")
        self.out, self.n = torch.zeros(12, 5, **i32), torch.zeros(12, **i32)
        self.data = torch.randn(2, 2, 90, 2, 16, 64, generator=g, device="cuda").bfloat16()
        self.pool = PagePool(self.data[:, 0], self.data[:, 1], torch.full((13, 6), -1, **i32), torch.zeros(13, **i32),
                             torch.zeros(90, **i32))
        self.status = torch.zeros(1, **i32)
        self.ws = torch.empty(self.pool.workspace(), **u8)
        reserve_pages(self.pool, torch.tensor([37], **i32), seq=torch.tensor([12], **i32))
        self.src, self.dst, self.rows = torch.full((12,), 12, **i32), torch.arange(12, **i32), torch.full((12,), 5, **i32)
        self.new, self.snap = torch.zeros(12, **i32), torch.zeros_like(self.data)

    def run(self, side):
        import torch
        from block_diffusion_speculative_hidden_gb300 import (compact_pages, fork_pages, gemm_fp4, quantize_fp4, reserve_pages,
                                                              truncate_pages, verify_tokens)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            fork_pages(self.pool, self.src, self.dst, workspace=self.ws, status=self.status)
            reserve_pages(self.pool, self.rows, seq=self.dst, workspace=self.ws, status=self.status)
        quantize_fp4(self.x, "nv", out=self.t)
        gemm_fp4(self.W, self.t, out=self.logits, status=self.status)
        torch.softmax(self.logits.view(12, 5, 1500), -1, out=self.p)
        verify_tokens(self.tok, self.p, self.ua, self.us, out=self.out, n_out=self.n, status=self.status)
        main.wait_stream(side)
        torch.add(self.n, 37, out=self.new)
        truncate_pages(self.pool, self.new, seq=self.dst, status=self.status)
        compact_pages(self.pool, workspace=self.ws, status=self.status)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            self.snap.copy_(self.data)
        self.x.add_(self.logits[:, :512].bfloat16())
        self.logits.fill_(float("nan"))
        main.wait_stream(side)

    def state(self):
        return [self.x, self.t.codes, self.p, self.out, self.n, self.data, self.snap, self.pool.page_table, self.pool.seq_len,
                self.pool.refs, self.status]


def test_two_streams():
    import torch
    a, b, c = Work(), Work(), Work()
    side = torch.cuda.Stream()
    for w in (a, b, c):
        w.run(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(side)
    for _ in range(6):
        a.run(side)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):                # the same step with the streams' parts exchanged
            side.wait_stream(torch.cuda.default_stream())
            b.run(torch.cuda.default_stream())
        torch.cuda.default_stream().wait_stream(side)
        g.replay()
        torch.cuda.synchronize()
        for x, y, z in zip(a.state(), b.state(), c.state()):
            assert torch.equal(x, y) and torch.equal(x, z)
        assert int(a.status.item()) == 0
