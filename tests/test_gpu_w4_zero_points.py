"""dflash_gemm_w4 with zero points over all of a byte: the differences code - zero enter the
product exactly, whatever the activations' type and the kernel that the row count selects."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["bfloat16", "float16"])
@pytest.mark.parametrize("M", [1, 12, 20, 32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_zero_point_exactly(x, M, group):
    """Activations that are 1 at one place of a group and 0 elsewhere, scales of 1: each output is one
    difference, an integer of at most 255, which nothing has to round."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    N, K = 256, 4 * group
    g = torch.Generator(device="cuda").manual_seed(M + group)
    W = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    zero = (torch.arange(N, device="cuda")[:, None] + 37 * torch.arange(4, device="cuda")).to(torch.uint8)
    scale = torch.ones(N, 4, device="cuda")
    codes = torch.stack([W & 15, W >> 4], -1).reshape(N, K).double()
    w = codes - zero.double().repeat_interleave(group, 1)
    for step in range(4):
        X = torch.zeros(M, K, device="cuda", dtype=getattr(torch, x))
        at = (torch.arange(M, device="cuda") * 41 + step * group + 7 * step) % K
        X[torch.arange(M, device="cuda"), at] = 1.0
        out = gemm_w4(W, scale, X, zero=zero.contiguous(), group=group)
        assert torch.equal(out.double(), w[:, at].t())


@pytest.mark.parametrize("x", ["bfloat16", "float16"])
@pytest.mark.parametrize("M,K,scale", [(1, 4096, "bfloat16"), (16, 1056, "float16"), (32, 2048, "float32")])
def test_products_with_large_zero_points(x, M, K, scale):
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    from decode_ref import check_w4
    g = torch.Generator(device="cuda").manual_seed(5)
    N, group = 600, 64
    gs = -(-K // group)
    W = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sc = (torch.rand(N, gs, generator=g, device="cuda") * 0.02 + 0.001).to(getattr(torch, scale))
    z = torch.randint(0, 256, (N, gs), generator=g, device="cuda", dtype=torch.uint8)
    X = torch.randn(M, K, generator=g, device="cuda").to(getattr(torch, x))
    check_w4(gemm_w4(W, sc, X, zero=z, group=group), W, sc, X, z, group, "int4")
