"""Sizes of dflash_gemm_w4 whose counts would not fit 32 bits are refused on the host (addresses that
are never followed)."""
import pytest

UNSUPPORTED = 2
P = 1 << 20


@pytest.fixture(scope="module")
def L():
    from block_diffusion_speculative_hidden_gb300 import _lib, build_lib
    build_lib.build()
    return _lib.lib()


@pytest.mark.parametrize("N,K,M", [
    (16, 1 << 26, 16),               # 16 rows of activations of 2 K bytes: 2^31 bytes of them
    (1, 1 << 30, 1), (1, (1 << 31) - 32, 1), (16, (1 << 26) + 32, 32), ((1 << 31) - 1, 32, 1), ((1 << 31) - 5, 64, 20)])
@pytest.mark.parametrize("fmt,group", [(0, 32), (1, 128)])
def test_counts_past_32_bits(L, N, K, M, fmt, group):
    assert L.dflash_gemm_w4(P, fmt, P, 1, None, N, K, group, P, 1, M, P, None, None) == UNSUPPORTED


def test_shared_memory_plan_stays_within_32_bits():
    """What the largest allowed call asks of the resident kernel's plan: 2 bytes an activation of all of k,
    rounded up to units of 256, and 64 bytes a row."""
    for M in range(1, 17):
        K = (1 << 29) // M // 32 * 32
        units = -(-K // 256)
        assert M * (units * 512 + 64) + 1023 < 1 << 31
