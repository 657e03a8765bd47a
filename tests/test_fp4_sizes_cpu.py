"""Matrices of 4-bit floats whose row would not fit 32 bits are refused when they are made (tensors without memory)."""
import pytest


def _tiles(rows, cols, fmt):
    return -(-rows // 128) * -(-cols // 256) * (2048 if fmt == "nv" else 1024)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("cols", [2 ** 31, 2 ** 32, 2 ** 32 + 64, 2 ** 33 + 4096])
def test_columns_past_32_bits(fmt, cols):
    import torch
    from block_diffusion_speculative_hidden_gb300 import Fp4
    codes = torch.empty(1, cols // 2, dtype=torch.uint8, device="meta")
    scales = torch.empty(_tiles(1, cols, fmt), dtype=torch.uint8, device="meta")
    with pytest.raises(ValueError, match="columns"):
        Fp4(codes, scales, fmt)
    with pytest.raises(ValueError, match="columns"):
        Fp4._empty(1, cols, fmt, None, -1, torch.device("meta"))
