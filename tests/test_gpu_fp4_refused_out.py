"""A quantising call that is refused leaves the matrix that it should have written as it was."""
import pytest

pytestmark = pytest.mark.gpu


def test_a_refused_call_keeps_the_scale():
    import torch
    from block_diffusion_speculative_hidden_gb300 import DflashError, Fp4, quantize_fp4
    x = torch.randn(4, 64, device="cuda")
    raw, scales = torch.zeros(4 * 32 + 16, dtype=torch.uint8, device="cuda"), torch.zeros(2048, dtype=torch.uint8, device="cuda")
    old, new = torch.full((1,), 0.5, device="cuda"), torch.full((1,), 0.25, device="cuda")
    odd = Fp4(raw[8:8 + 128].view(4, 32), scales, "nv", old)      # codes at 8 bytes: refused by the library
    at = odd.at
    for scale in (new, None):
        with pytest.raises(DflashError):
            quantize_fp4(x, "nv", scale=scale, out=odd)
        assert odd.at == at and odd.scale.data_ptr() == old.data_ptr()
    good = Fp4(raw[:128].view(4, 32), scales, "nv", old)
    assert quantize_fp4(x, "nv", scale=new, out=good) is good
    assert good.scale.data_ptr() == new.data_ptr() == good.at[2]
    quantize_fp4(x, "nv", out=good)
    assert good.scale is None and good.at[2] is None
