"""The batch operators on memory at the least alignment that they take: pages, codes, scales and outputs at 16 bytes."""
import pytest

pytestmark = pytest.mark.gpu


def _at(n, dtype, bytes_off):
    """n entries of dtype that start bytes_off behind a 256-byte boundary."""
    import torch
    size = torch.empty(0, dtype=dtype).element_size()
    room = torch.empty(n + 256, dtype=dtype, device="cuda")
    first = (-room.data_ptr() % 256 + bytes_off) // size
    t = room[first:first + n]
    assert t.data_ptr() % 256 == bytes_off
    return t


@pytest.mark.parametrize("off", [0, 16, 32, 48])
@pytest.mark.parametrize("dtype,dh,Hkv,layers", [("float16", 64, 3, 2), ("float32", 32, 1, 9), ("bfloat16", 128, 2, 1)])
def test_pages(off, dtype, dh, Hkv, layers):
    import torch
    from block_diffusion_speculative_hidden_gb300 import PagePool, compact_pages, copy_pages, fork_pages, reserve_pages
    n, dt = 40, getattr(torch, dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    k, v = ([_at(n * Hkv * 16 * dh, dt, off).view(n, Hkv, 16, dh) for _ in range(layers)] for _ in range(2))
    for t in [*k, *v]:
        t.copy_(torch.randn(t.shape, device="cuda"))
    k0, v0 = [t.clone() for t in k], [t.clone() for t in v]
    pool = PagePool(k, v, torch.full((5, 6), -1, **i32), torch.zeros(5, **i32), torch.zeros(n, **i32))
    status = torch.zeros(1, **i32)

    def same(pairs):
        for a, b in zip([*k, *v], [*k0, *v0]):
            for dst, src in pairs:
                assert torch.equal(a[dst], b[src]), (dst, src)
    reserve_pages(pool, torch.tensor([40, 90], **i32), status=status)
    assert pool.page_table[:2, :6].tolist() == [[0, 1, 2, -1, -1, -1], [3, 4, 5, 6, 7, 8]]
    fork_pages(pool, torch.tensor([0, 1], **i32), torch.tensor([2, 3], **i32), status=status)
    same([(9, 2), (10, 8), (2, 2), (8, 8)])
    reserve_pages(pool, torch.tensor([1], **i32), seq=torch.tensor([3], **i32), status=status)   # its own page: no copy
    copy_pages(pool, torch.tensor([1, 2, 30], **i32), torch.tensor([39, 38, 37], **i32), status=status)
    same([(39, 1), (38, 2), (37, 30), (36, 36)])
    pool.refs[39] = 1
    compact_pages(pool, status=status)
    same([(11, 1), (38, 2)])
    assert int(status.item()) == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dt", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("off", [16, 32, 48])
def test_taken_back(fmt, dt, off):
    import torch
    from block_diffusion_speculative_hidden_gb300 import dequantize_fp4, quantize_fp4
    t = quantize_fp4(torch.randn(33, 288, generator=torch.Generator("cuda").manual_seed(3), device="cuda"), fmt)
    out = _at(33 * 288, getattr(torch, dt), off).view(33, 288)
    assert dequantize_fp4(t, out=out) is out
    assert torch.equal(out, dequantize_fp4(t, out.dtype))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
# (one CTA a tile, shared tiles, pairs, many tiles)
@pytest.mark.parametrize("M,N,K", [(40, 640, 320), (16, 128, 4096), (640, 4096, 512), (240, 32768, 256)])
@pytest.mark.parametrize("off", [16, 48, 112])
def test_products(fmt, M, N, K, off):
    import torch
    from block_diffusion_speculative_hidden_gb300 import Fp4, gemm_fp4, quantize_fp4
    g = torch.Generator("cuda").manual_seed(M)
    ops = [quantize_fp4(torch.randn(r, K, generator=g, device="cuda"), fmt) for r in (N, M)]
    want = gemm_fp4(*ops)

    def moved(t):
        codes, scales = _at(t.codes.numel(), torch.uint8, off), _at(t.scales.numel(), torch.uint8, off)
        return Fp4(codes.copy_(t.codes.flatten()).view(t.codes.shape), scales.copy_(t.scales.flatten()), fmt)
    out = _at(M * N, torch.bfloat16, off).view(M, N)
    gemm_fp4(moved(ops[0]), moved(ops[1]), out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantised(fmt):
    import torch
    from block_diffusion_speculative_hidden_gb300 import Fp4, quantize_fp4
    x = _at(65 * 320, torch.bfloat16, 32).view(65, 320)
    x.copy_(torch.randn(65, 320, device="cuda"))
    want = quantize_fp4(x, fmt)
    for off in (16, 48):
        y = _at(65 * 320, torch.bfloat16, off).view(65, 320).copy_(x)
        out = Fp4(_at(65 * 160, torch.uint8, off).view(65, 160), _at(want.scales.numel(), torch.uint8, off), fmt)
        out.scales.copy_(want.scales)
        quantize_fp4(y, fmt, out=out)
        assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
