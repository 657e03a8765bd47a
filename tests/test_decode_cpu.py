"""What the decode-step operators refuse on the host, through the C ABI with
addresses that are never followed, and through the Python faces."""
import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
P = 1 << 20        # an aligned address; nothing is enqueued in these calls


@pytest.fixture(scope="module")
def L():
    from block_diffusion_speculative_hidden_gb300 import _lib, build_lib
    build_lib.build()
    return _lib.lib()


def _kv(**kw):
    from block_diffusion_speculative_hidden_gb300 import _lib
    a = dict(k=P, v=P, page_table=P, seq_len=P, n_pages=100, n_seqs=5, max_pages=20, n_kv_heads=2, head_dim=64, elem=1)
    a.update(kw)
    return _lib.DflashPagedKV(*a.values())


BAD_KV = [dict(k=None), dict(v=None), dict(page_table=None), dict(seq_len=None), dict(n_pages=0), dict(n_seqs=0),
          dict(max_pages=0), dict(n_kv_heads=0), dict(head_dim=0), dict(elem=3), dict(elem=-1), dict(k=P + 8),
          dict(v=P + 2), dict(max_pages=1 << 30)]


def _append(L, kv=None, **kw):
    a = dict(k=P, ld_k=128, v=P, ld_v=128, src=1, n_rows=None, seq=None, base=None, B=3, T=2, cos=P, sin=P, rows=64,
             q=P, ld_q=256, Hq=4, q_out=P, status=None, stream=None)
    a.update(kw)
    return L.dflash_append_kv(ctypes.byref(kv if kv is not None else _kv()), *a.values())


def test_append_refusals(L):
    for bad in BAD_KV:
        assert _append(L, _kv(**bad)) == INVALID, bad
    assert L.dflash_append_kv(None, *([None, 0] * 2), 1, None, None, None, 1, 1, None, None, 0, None, 0, 0, None, None,
                              None) == INVALID
    for bad in (dict(k=None), dict(v=None), dict(B=0), dict(T=0), dict(src=3), dict(src=-1), dict(cos=None),
                dict(sin=None), dict(rows=0), dict(cos=P + 4), dict(sin=P + 8), dict(q=None), dict(q_out=None),
                dict(Hq=0), dict(q_out=P + 8), dict(ld_k=127), dict(ld_v=64), dict(ld_q=255), dict(k=P + 1),
                dict(v=P + 1), dict(q=P + 1), dict(B=6), dict(Hq=1 << 30)):
        assert _append(L, **bad) == INVALID, bad
    assert _append(L, src=0, k=P + 2) == INVALID
    assert _append(L, _kv(head_dim=96), ld_k=192, ld_v=192, ld_q=400) == UNSUPPORTED
    assert _append(L, B=5, T=(1 << 31) - 1) == UNSUPPORTED


def _attend(L, kv=None, **kw):
    a = dict(q=P, ld_q=256, Hq=4, n_rows=None, seq=None, B=3, T=2, off=P, pre=P, NG=1, causal=1, scale=0.0,
             max_prefix=0, max_len=0, out=2 * P, lse=None, ws=P, ws_bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    return L.dflash_prefix_attention(ctypes.byref(kv if kv is not None else _kv()), *a.values())


def test_attention_refusals(L):
    for bad in BAD_KV:
        assert _attend(L, _kv(**bad)) == INVALID, bad
    for bad in (dict(q=None), dict(out=None), dict(ws=None), dict(B=0), dict(T=0), dict(NG=-1), dict(off=None),
                dict(pre=None), dict(NG=0), dict(Hq=0), dict(Hq=5), dict(ld_q=255), dict(ld_q=252), dict(ld_q=248),
                dict(q=P + 8), dict(out=P + 8), dict(ws=P + 128), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(max_prefix=-1), dict(max_len=-1), dict(B=6),
                dict(out=P, ld_q=264)):
        assert _attend(L, **bad) == INVALID, bad
    assert _attend(L, _kv(elem=0)) == UNSUPPORTED                  # fp32 caches
    assert _attend(L, _kv(head_dim=32)) == UNSUPPORTED
    assert _attend(L, _kv(head_dim=96), ld_q=400) == UNSUPPORTED
    assert _attend(L, T=1 << 29) == UNSUPPORTED
    assert _attend(L, B=4097, seq=P) == UNSUPPORTED and _attend(L, NG=4097) == UNSUPPORTED
    assert _attend(L, ws_bytes=255) == WORKSPACE


def test_attention_workspace(L):
    def size(kv=None, Hq=4, B=3, T=2, NG=1, mp=0, ml=0):
        return L.dflash_prefix_attention_workspace(ctypes.byref(kv if kv is not None else _kv()), Hq, B, T, NG, mp, ml)
    assert size() > 0 and size(NG=0) > 0
    # partial results in fp32: at least one prefix and one own part per row
    assert size(mp=100, ml=100) >= 2 * 3 * 2 * 4 * (64 + 1) * 4
    for bad in (dict(Hq=5), dict(B=0), dict(T=0), dict(NG=-1), dict(mp=-1), dict(kv=_kv(elem=0)), dict(T=1 << 29)):
        assert size(**bad) == 0, bad
    need = size()
    assert _attend(L, ws_bytes=need - 1) == WORKSPACE


def _w4(L, **kw):
    a = dict(W=P, fmt=0, scale=P, se=1, zero=None, N=64, K=128, group=32, X=P, xe=1, M=1, out=P, status=None,
             stream=None)
    a.update(kw)
    return L.dflash_gemm_w4(*a.values())


def test_w4_refusals(L):
    for bad in (dict(W=None), dict(scale=None), dict(X=None), dict(out=None), dict(N=0), dict(K=0), dict(M=0),
                dict(fmt=2), dict(fmt=-1), dict(fmt=1, zero=P), dict(se=3), dict(xe=0), dict(xe=3), dict(W=P + 8),
                dict(X=P + 8), dict(scale=P + 1), dict(se=0, scale=P + 2), dict(out=P + 2)):
        assert _w4(L, **bad) == INVALID, bad
    for bad in (dict(M=33), dict(K=48), dict(group=16), dict(group=256), dict(group=0)):
        assert _w4(L, **bad) == UNSUPPORTED, bad


def test_table_and_extend_refusals(L):
    assert L.dflash_rope_table(None, P, 4, 64, 1e4, None) == INVALID
    assert L.dflash_rope_table(P, None, 4, 64, 1e4, None) == INVALID
    assert L.dflash_rope_table(P, P, 0, 64, 1e4, None) == INVALID
    assert L.dflash_rope_table(P, P, 4, 64, 0.0, None) == INVALID
    assert L.dflash_rope_table(P, P, 4, 96, 1e4, None) == UNSUPPORTED
    assert L.dflash_rope_table(P, P, 1 << 30, 128, 1e4, None) == UNSUPPORTED
    assert L.dflash_extend(None, P, 0, 1, 1, None) == INVALID


def test_python_faces_refuse():
    import torch
    from block_diffusion_speculative_hidden_gb300 import PagedKV, append_kv, gemm_w4, prefix_attention
    i32 = torch.int32
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    for bad in (lambda: PagedKV(k, k[:, :1], table, lens), lambda: PagedKV(k, k.half(), table, lens),
                lambda: PagedKV(k[:, :, :8], k[:, :, :8], table, lens), lambda: PagedKV(k, k, table.long(), lens),
                lambda: PagedKV(k, k, table, lens[:2]), lambda: PagedKV(k.double(), k.double(), table, lens),
                lambda: PagedKV(k.transpose(0, 1), k, table, lens), lambda: PagedKV(k, k, table.t(), lens)):
        with pytest.raises(ValueError):
            bad()
    kv = PagedKV(k, k, table, lens)
    x = torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 1, 4, 64, dtype=torch.bfloat16)
    W, s, X = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2), torch.zeros(1, 64, dtype=torch.bfloat16)
    for bad in (lambda: append_kv(kv, x, x),                                   # a cache that is not on a CUDA device
                lambda: append_kv(kv, x[..., :32], x[..., :32]), lambda: append_kv(kv, x, x.half()),
                lambda: append_kv(kv, x[:, :, :1], x[:, :, :1]), lambda: prefix_attention(kv, q),
                lambda: prefix_attention(kv, q.half()), lambda: prefix_attention(kv, q, lens),
                lambda: gemm_w4(W, s, X, group=32), lambda: gemm_w4(W, s, X, group=0),
                lambda: gemm_w4(W, s, X.float(), group=32), lambda: gemm_w4(W, s[:, :1], X, group=32),
                lambda: gemm_w4(W, s, X, group=32, fmt="nf4"), lambda: gemm_w4(W.int(), s, X, group=32),
                lambda: gemm_w4(W, s, X[:, :32].contiguous(), group=32)):
        with pytest.raises(ValueError):
            bad()
