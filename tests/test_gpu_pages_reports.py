"""What a call that asks for too many pages reports when an entry far behind is wrong as well."""
import pytest

pytestmark = pytest.mark.gpu

EXHAUSTED, TOO_LONG, BAD_ROWS, BAD_PAGE = 1, 2, 16, 64


@pytest.mark.parametrize("at", [3, 600, 1100, 1499])
def test_a_wrong_entry_comes_before_missing_pages(at):
    from block_diffusion_speculative_hidden_gb300 import reserve_pages
    from pages_ref import Pool
    from test_gpu_pages import _grow
    n = 1500
    P = Pool(300, n, 8, layers=1, Hkv=1, dh=32)
    _grow(P, [5] + [0] * (n - 1))
    for rows, bit in ((1, EXHAUSTED), (-1, BAD_ROWS), (129, TOO_LONG), (2 ** 31 - 1, TOO_LONG), (128, EXHAUSTED)):
        want = [100] * n
        want[at] = rows
        old = P.frozen()
        reserve_pages(P.pool, P.ints(want), status=P.status)
        assert int(P.status.item()) == bit and P.unchanged(old), (rows, bit)
        P.status.zero_()
    P.lens[at] = 7                                   # a sequence whose page is not there
    old = P.frozen()
    reserve_pages(P.pool, P.ints([100] * n), status=P.status)
    assert int(P.status.item()) == BAD_PAGE and P.unchanged(old)
    P.status.zero_()
    P.lens[at] = 0
    few = [0] * n                                    # as many as there are, the last ones far behind
    few[0], few[1100:1109], few[1499] = 11, [128] * 9, 16 * 6
    reserve_pages(P.pool, P.ints(few), status=P.status)
    P.m.reserve(range(n), few)
    P.check()
