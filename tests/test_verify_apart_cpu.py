"""Verification refuses outputs that lie over its inputs or each other (addresses that are never followed)."""
import pytest

INVALID = 1
A = 1 << 24


@pytest.fixture(scope="module")
def L():
    from block_diffusion_speculative_hidden_gb300 import _lib, build_lib
    build_lib.build()
    return _lib.lib()


@pytest.mark.parametrize("te,de", [(0, 1), (2, 0)])
def test_outputs_over_inputs_are_refused(L, te, de):
    B, K, V, ld_t, ld_d = 3, 4, 100, 104, 112
    ts, ds = (4, 2, 2)[te], (4, 2, 2)[de]
    base = dict(tokens=A, n=2 * A, target=3 * A, te=te, ld_t=ld_t, draft=4 * A, de=de, ld_d=ld_d, ua=5 * A, us=6 * A, B=B, K=K, V=V,
                out=7 * A, n_out=8 * A, status=9 * A, stream=None)
    size = dict(tokens=4 * B * K, n=4 * B, target=((B * (K + 1) - 1) * ld_t + V) * ts, draft=((B * K - 1) * ld_d + V) * ds,
                ua=4 * B * K, us=4 * B, out=4 * B * (K + 1), n_out=4 * B, status=4)
    for o in ("out", "n_out", "status"):
        for i in size:
            if i == o:
                continue
            for at in (base[i], base[i] + (size[i] - 1) // 4 * 4, base[i] - size[o] + 4):
                assert L.dflash_verify_tokens(*{**base, o: at}.values()) == INVALID, (o, i, at - base[i])
