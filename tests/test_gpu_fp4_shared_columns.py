"""Products whose CTAs have several tiles and accumulators that share TMEM columns: heights whose last block of 32
rows is a half, many tiles a CTA, again and again."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("M,N,K", [(225, 32768, 1024), (239, 50000, 1024), (240, 32768, 2048), (161, 50000, 544),
                                   (176, 32768, 1024), (193, 32768, 1024), (208, 50000, 288), (256, 32768, 1024)])
def test_halves_of_the_last_block(M, N, K, dt):
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_fp4
    from fp4_ref import check_product
    from test_gpu_fp4 import _operand
    # (fp16: sums below 36 * 448^2 * 2048 / 2^20 < 2^14)
    g = (2.0 ** -10, 2.0 ** -10)
    W, w = _operand(N, K, "nv", M, g=g[0])
    X, x = _operand(M, K, "nv", M + 1, g=g[1])
    out = torch.empty(M, N, dtype=getattr(torch, dt), device="cuda")
    gemm_fp4(W, X, out=out)
    check_product(out, w, x, g[0] * g[1])
    for _ in range(20):
        again = gemm_fp4(W, X, dtype=out.dtype)
        assert torch.equal(out, again)
