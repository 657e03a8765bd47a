"""Cuts to lengths next to 2^31, which keep all of a sequence, beside real ones."""
import pytest

pytestmark = pytest.mark.gpu

FAR = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 15, 2 ** 31 - 16, 2 ** 31 - 17, 2 ** 30, 2 ** 27]


def _cut(P, seq, new):
    from block_diffusion_speculative_hidden_gb300 import truncate_pages
    truncate_pages(P.pool, P.ints(new), seq=P.ints(seq), status=P.status)


@pytest.mark.parametrize("far", FAR)
def test_a_far_length_keeps_all(far):
    from pages_ref import Pool
    from test_gpu_pages import _grow
    P = Pool(60, 8, 9)
    _grow(P, [40, 16, 0, 129, 144, 1])
    seq, new = [4, 0, 1, 2, 3, 5], [far, 17, far, far, far, 0]
    _cut(P, seq, new)
    P.m.truncate(seq, new)
    P.check()
    _cut(P, [0, 1, 2, 3, 4, 5], [far] * 6)
    P.check()


def test_many_far_lengths():
    """More entries than are staged, every other one cut; pages that others hold too."""
    from block_diffusion_speculative_hidden_gb300 import fork_pages
    from pages_ref import Pool
    from test_gpu_pages import _grow
    n = 1500
    P = Pool(4000, n, 8, layers=1, Hkv=1, dh=32)
    _grow(P, [100, 33])
    src, dst = [i % 2 for i in range(n - 2)], list(range(2, n))
    fork_pages(P.pool, P.ints(src), P.ints(dst), status=P.status)
    P.m.fork(src, dst)
    new = [FAR[i % len(FAR)] if i % 2 else i % 100 for i in range(n)]
    _cut(P, list(range(n)), new)
    P.m.truncate(range(n), new)
    P.check()


def test_a_far_length_looks_at_nothing_that_it_keeps():
    """Entries of the table in front of the kept length are not looked at, whatever they hold."""
    import torch
    from pages_ref import Pool
    from test_gpu_pages import _grow
    P = Pool(20, 3, 5)
    _grow(P, [40, 20])
    P.table[0, 1] = 10 ** 9
    old = P.frozen()
    _cut(P, [0], [2 ** 31 - 1])
    assert int(P.status.item()) == 0 and P.unchanged(old)
    _cut(P, [0], [-2 ** 31])
    assert int(P.status.item()) & 16 and P.unchanged(old)
    torch.cuda.synchronize()
