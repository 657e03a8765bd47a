"""The lengths themselves as numbers of a call, and the pool's own table and counts as outputs."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [5, 1300])
def test_lengths_as_numbers(n):
    from block_diffusion_speculative_hidden_gb300 import compact_pages, reserve_pages, truncate_pages
    from pages_ref import Pool
    from test_gpu_pages import _grow
    P = Pool(7 * n, n, 9, layers=1, Hkv=1, dh=32)
    _grow(P, [(13 * i) % 50 for i in range(n)])
    truncate_pages(P.pool, P.lens, status=P.status)                  # nothing
    P.check()
    reserve_pages(P.pool, P.lens, status=P.status)                   # twice as long
    P.m.reserve(range(n), list(P.m.lens))
    P.check()
    reserve_pages(P.pool, P.lens[:3], status=P.status)
    P.m.reserve(range(3), P.m.lens[:3])
    P.check()
    gone = list(range(0, n, 2))
    truncate_pages(P.pool, seq=P.ints(gone), status=P.status)
    P.m.truncate(gone, [0] * len(gone))
    compact_pages(P.pool, table_out=P.table, refs_out=P.refs, status=P.status)
    P.m.compact()
    P.check()
    for bad in (lambda: truncate_pages(P.pool, P.lens[:2], seq=P.ints([1, 0])), lambda: reserve_pages(P.pool, P.lens[1:3]),
                lambda: truncate_pages(P.pool, seq=P.refs[:3]), lambda: compact_pages(P.pool, page_map=P.refs)):
        from block_diffusion_speculative_hidden_gb300 import DflashError
        with pytest.raises(DflashError):
            bad()
    P.check()
