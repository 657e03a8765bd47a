"""NV scale bytes with the sign bit, which are no steps: taken back and multiplied alike."""
import pytest

pytestmark = pytest.mark.gpu


def test_signed_bytes_are_no_steps():
    import torch
    from block_diffusion_speculative_hidden_gb300 import Fp4, dequantize_fp4, gemm_fp4, quantize_fp4
    rows, K = 256, 64
    codes = torch.randint(0, 256, (rows, K // 2), generator=torch.Generator().manual_seed(1)).to(torch.uint8).cuda()
    sc = torch.full((rows, K // 16), 56, dtype=torch.uint8)
    sc[:, 2] = torch.arange(rows).to(torch.uint8)
    t = Fp4.from_rows(codes, sc.cuda(), "nv")
    bad = torch.zeros(rows, K, dtype=torch.bool)
    bad[127, 32:48] = True
    bad[129:, 32:48] = True                          # (-0 is a step of 0)
    v = dequantize_fp4(t, torch.float32).cpu()
    assert torch.equal(torch.isnan(v), bad)
    assert (v[128, 32:48] == 0).all()
    w = torch.randn(33, K, generator=torch.Generator().manual_seed(2)).cuda()
    for out in (gemm_fp4(quantize_fp4(w, "nv"), t, dtype=torch.float32), gemm_fp4(t, quantize_fp4(w, "nv"), dtype=torch.float32).t()):
        assert torch.equal(torch.isnan(out).any(1).cpu(), bad.any(1)) and torch.equal(torch.isnan(out).all(1).cpu(), bad.any(1))
    # the same bytes in the tiles themselves
    raw = quantize_fp4(w[:1].expand(128, K).contiguous(), "nv")
    for b in (128, 129, 200, 254, 255):
        raw.scales[0] = b
        v = dequantize_fp4(raw, torch.float32)
        assert (v[0, :16] == 0).all() if b == 128 else torch.isnan(v[0, :16]).all()
        assert torch.isfinite(v[1:]).all() and torch.isfinite(v[0, 16:]).all()
