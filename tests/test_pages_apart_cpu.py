"""Page calls refuse arrays that lie over the pool's or over their workspace (addresses that are never followed)."""
import ctypes

import pytest

INVALID = 1
A = 1 << 24
SEQS, MAX, PAGES = 5, 20, 100
TABLE, LENS, REFS, WS, FREE = A, 2 * A, 3 * A, 4 * A, 5 * A


@pytest.fixture(scope="module")
def L():
    from block_diffusion_speculative_hidden_gb300 import _lib, build_lib
    build_lib.build()
    return _lib.lib()


def _pool():
    from block_diffusion_speculative_hidden_gb300 import _lib
    k = (ctypes.c_void_p * 1)(8 * A)
    return _lib.DflashPagePool(k, k, TABLE, LENS, REFS, 1, PAGES, SEQS, MAX, 2, 64, 1)


def _overlaps(n, ws):
    """Addresses of n int32 that meet the first or the last entry of an array of the pool's, or of the workspace."""
    at = [(TABLE, SEQS * MAX), (LENS, SEQS), (REFS, PAGES)] + ([(WS, ws // 4)] if ws else [])
    return [x for a, size in at for x in (a, a + 4, a - 4 * (n - 1), a + 4 * (size - 1))]


def test_arrays_over_the_pools_are_refused(L):
    pool = _pool()
    need = L.dflash_pages_workspace(ctypes.byref(pool))
    B = 3
    fork = dict(src=FREE, dst=FREE + 64, B=B, ws=WS, size=need, status=FREE + 128, stream=None)
    cut = dict(seq=FREE, new=FREE + 64, B=B, status=FREE + 128, stream=None)
    room = dict(seq=FREE, rows=FREE + 64, B=B, ws=WS, size=need, status=FREE + 128, stream=None)
    pack = dict(table=FREE, refs=FREE + 4096, map=FREE + 8192, n=FREE + 16384, ws=WS, size=need, status=FREE + 20000, stream=None)
    sizes = dict(src=B, dst=B, seq=B, new=B, rows=B, status=1, table=SEQS * MAX, refs=PAGES, map=PAGES, n=1)
    for f, base in ((L.dflash_pages_fork, fork), (L.dflash_pages_truncate, cut), (L.dflash_pages_reserve, room),
                    (L.dflash_pages_compact, pack)):
        for name in set(base) & set(sizes):
            for x in _overlaps(sizes[name], need if "ws" in base else 0):
                if (name, x) in (("table", TABLE), ("refs", REFS)):
                    continue                         # the pool's own as outputs
                assert f(ctypes.byref(pool), *{**base, name: x}.values()) == INVALID, (f, name, x)
        if "ws" in base:
            for x in (TABLE, LENS, REFS, REFS - need + 16, TABLE + 4 * SEQS * MAX - 16):
                assert f(ctypes.byref(pool), *{**base, "ws": x}.values()) == INVALID, (f, x)
    # the lengths as numbers of a call: only entry i for sequence i
    assert L.dflash_pages_truncate(ctypes.byref(pool), FREE, LENS, B, None, None) == INVALID
    assert L.dflash_pages_truncate(ctypes.byref(pool), None, LENS + 4, B, None, None) == INVALID
    assert L.dflash_pages_reserve(ctypes.byref(pool), FREE, LENS, B, WS, need, None, None) == INVALID
