"""dflash_prefix_attention against softmax attention in 64 bits: head layouts,
one token to 17, lengths of zero and one, pages that end inside a tile, groups
(none, several, empty, without a prefix), causal and unmasked blocks, rows that
see nothing, uneven row counts, strided queries, NaN behind every length, a
cache past 32-bit offsets, recorded calls, and bad entries."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(B, T, Hq, Hkv, dh, dtype, own_lens, groups=(), n=None, causal=True, scale=0.0, seq=None, pad=0, seed=1,
         hints=True, want_lse=True, q_mul=2.0, in_place=False, **kw):
    """groups: [(entries, prefix length or None)].  Builds the cache, calls once, checks everything."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache, check_attention
    dt = getattr(torch, dtype)
    rows = list(own_lens)
    off, pre, spans = [0], [], []
    for count, length in groups:
        spans.append((off[-1], off[-1] + count, len(rows) if length is not None else -1))
        pre.append(len(rows) if length is not None else -1)
        off.append(off[-1] + count)
        if length is not None:
            rows.append(length)
    assert not groups or off[-1] == B
    c = Cache(rows, Hkv, dh, dt, seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    width = Hq * dh + pad
    q = (torch.randn(B, T, width, generator=g, device="cuda") * q_mul).to(dt)[:, :, :Hq * dh].unflatten(2, (Hq, dh))
    q0 = q.clone()
    out = q if in_place else torch.full((B, T, Hq, dh), 7.0, dtype=dt, device="cuda")
    lse = torch.full((B, T, Hq), 7.0, device="cuda") if want_lse else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    own = list(range(B)) if seq is None else seq
    nr = [T] * B if n is None else n
    prefix_attention(c.paged(), q, _ints(off) if groups else None, _ints(pre) if groups else None,
                     None if n is None else _ints(n), seq=None if seq is None else _ints(seq), causal=causal,
                     scale=scale, max_prefix=max([l for _, l in groups if l] + [1]) if hints and groups else 0,
                     max_len=max(max(own_lens), 1) if hints else 0, out=out, lse=lse, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    s = scale if scale else 1.0 / math.sqrt(dh)
    checked = check_attention(c, q0, out, lse, nr, own, spans, causal, s)
    assert checked == sum(nr)
    for b in range(B):                       # rows behind the last one stay
        if not in_place:
            assert (out[b, nr[b]:] == 7.0).all()
        assert lse is None or (lse[b, nr[b]:] == 7.0).all()
    return c, q0, out, lse


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 4), (6, 2), (8, 2), (10, 2), (16, 2), (12, 1), (32, 1)])
def test_head_layouts(dtype, dh, Hq, Hkv):
    _run(3, 1, Hq, Hkv, dh, dtype, [1, 33, 200], [(3, 77)])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 40])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_per_entry(dtype, T, causal):
    _run(4, T, 8, 2, 128, dtype, [T, T + 1, T + 15, 300], [(1, 5), (3, 130)], causal=causal)


@pytest.mark.parametrize("P", [0, 1, 15, 16, 17, 127, 128, 129, 1000, 5003])
@pytest.mark.parametrize("dh", [64, 128])
def test_prefix_lengths(P, dh):
    _run(5, 3, 8, 2, dh, "bfloat16", [3, 4, 16, 17, 130], [(5, P)])


@pytest.mark.parametrize("L", [0, 1, 15, 16, 17, 31, 32, 63, 64, 65, 127, 128, 129, 700, 4097])
def test_own_lengths_without_prefix(L):
    _run(2, 1, 8, 2, 128, "float16", [L, 5])
    _run(1, 1, 8, 2, 64, "bfloat16", [L])


def test_groups_of_every_kind():
    # prefixes of several lengths, a group without one, empty groups, an empty prefix
    _run(9, 4, 8, 2, 64, "float16", [4, 9, 0, 33, 100, 5, 1, 64, 17],
         [(0, 40), (3, 300), (1, None), (0, None), (2, 0), (3, 65)])


def test_rows_that_see_nothing():
    # more rows than own tokens, no prefix: the first rows see no key at all
    c, q, out, lse = _run(3, 6, 4, 2, 64, "bfloat16", [2, 0, 6], [(3, None)])
    assert (lse[0, :4] == -math.inf).all() and (out[0, :4] == 0).all() and (lse[1] == -math.inf).all()
    _run(3, 6, 4, 2, 128, "float16", [2, 0, 6])
    _run(2, 6, 4, 2, 128, "float16", [0, 0], [(2, 0)], causal=False)


def test_uneven_rows():
    _run(7, 17, 8, 2, 128, "bfloat16", [17, 3, 40, 0, 200, 16, 1], [(4, 90), (3, None)], n=[17, 3, 0, 5, 1, 16, 1])


def test_many_rows_on_one_prefix():
    _run(40, 17, 16, 2, 64, "float16", [17 + 7 * i for i in range(40)], [(40, 1100)])
    _run(21, 17, 8, 2, 128, "bfloat16", [17 + 31 * i for i in range(21)], [(13, 700), (8, 131)])


@pytest.mark.parametrize("dh", [64, 128])
def test_many_rows_and_keys(dh):
    """Several key tiles of a wide row tile, ragged against every tile edge."""
    for P in (255, 256, 257, 511, 513, 1025):
        _run(9, 17, 8, 2, dh, "bfloat16", [17, 20, 300, 17, 129, 128, 127, 640, 33], [(9, P)], seed=P)


def test_sharp_and_flat_scores():
    # one key dominates / all keys alike / scores far from zero, where a maximum moves late
    _run(4, 4, 8, 2, 128, "float16", [40, 500, 64, 4], [(4, 333)], q_mul=20.0)
    _run(4, 4, 8, 2, 128, "bfloat16", [40, 500, 64, 4], [(4, 333)], scale=1e-6)
    _run(33, 17, 8, 2, 64, "float16", [17 + i for i in range(33)], [(33, 1333)], q_mul=20.0)


def test_rising_scores():
    """Scores that rise along the keys: the running maximum moves at every tile."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache, check_attention
    for dh, T, B in ((64, 1, 2), (128, 17, 8), (64, 17, 8)):
        c = Cache([60] * B + [900], 2, dh, torch.float16, 5)
        for s in range(B + 1):
            i = torch.arange(c.lens[s], device="cuda")
            c.k[c.table[s].long()[i // 16], :, i % 16] = ((i + 900 * (s < B)) / 64.0).half()[:, None, None] * torch.ones(
                1, 2, dh, device="cuda", dtype=torch.float16)
        q = torch.ones(B, T, 8, dh, device="cuda", dtype=torch.float16)
        out, lse = torch.empty_like(q), torch.empty(B, T, 8, device="cuda")
        prefix_attention(c.paged(), q, _ints([0, B]), _ints([B]), out=out, lse=lse)
        check_attention(c, q, out, lse, [T] * B, list(range(B)), [(0, B, B)], True, 1 / math.sqrt(dh))


def test_strides_sequences_and_missing_hints():
    _run(3, 2, 8, 2, 64, "bfloat16", [70, 2, 9, 31, 5], [(3, 50)], seq=[4, 0, 3], pad=64, hints=False)
    _run(3, 1, 8, 2, 128, "float16", [70, 2, 9], [(1, 50), (2, 90)], seq=[1, 1, 0], pad=8, want_lse=False)


def test_in_place_output():
    _run(3, 5, 8, 2, 64, "float16", [70, 5, 9], [(3, 50)], in_place=True)
    _run(3, 5, 8, 2, 64, "float16", [70, 5, 9], in_place=True)
    _run(20, 17, 8, 2, 128, "bfloat16", [70 + i for i in range(20)], [(20, 200)], in_place=True)


def test_lengths_beyond_the_hints():
    """max_prefix and max_len only size the launch: longer contexts are attended in full."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache, check_attention
    c = Cache([900, 20, 3000], 2, 64, torch.float16, 4)
    q = torch.randn(2, 3, 8, 64, device="cuda", dtype=torch.float16)
    out, lse = torch.empty_like(q), torch.empty(2, 3, 8, device="cuda")
    prefix_attention(c.paged(), q, _ints([0, 2]), _ints([2]), max_prefix=1, max_len=1, out=out, lse=lse)
    check_attention(c, q, out, lse, [3, 3], [0, 1], [(0, 2, 2)], True, 1 / 8)


@pytest.mark.parametrize("T", [1, 17])
def test_offsets_past_32_bits(T):
    _run(3, T, 8, 8, 128, "bfloat16", [40, 17, 100], [(3, 200)], first_page=140000)


def test_long_prefix():
    _run(4, 1, 8, 2, 128, "float16", [1, 30, 100, 300], [(4, 70001)])
    _run(5, 17, 8, 1, 64, "bfloat16", [17, 30, 100, 300, 17], [(5, 20011)])


def test_same_result_every_time_and_on_any_stream():
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache
    c = Cache([70, 90, 17, 400, 2000], 2, 128, torch.bfloat16, 6)
    q = torch.randn(4, 17, 8, 128, device="cuda", dtype=torch.bfloat16)
    go, pre = _ints([0, 4]), _ints([4])
    first = prefix_attention(c.paged(), q, go, pre)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [prefix_attention(c.paged(), q, go, pre, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


def test_recorded_calls_follow_the_lengths():
    """Two recordings with a workspace each, replayed at the same time, with the lengths of the time."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention, prefix_attention_workspace
    from decode_ref import Cache, check_attention
    full = [200, 170, 900]
    c = Cache(full, 2, 64, torch.float16, 8)
    kv = c.paged()
    q = torch.randn(2, 1, 8, 64, device="cuda", dtype=torch.float16)
    go, pre = _ints([0, 2]), _ints([2])
    need = prefix_attention_workspace(kv, 8, 2, 1, 1, 900, 200)
    runs = []
    for _ in range(2):
        r = dict(ws=torch.empty(need, dtype=torch.uint8, device="cuda"), out=torch.zeros_like(q),
                 lse=torch.zeros(2, 1, 8, device="cuda"), graph=torch.cuda.CUDAGraph(), stream=torch.cuda.Stream())
        args = dict(max_prefix=900, max_len=200, out=r["out"], lse=r["lse"], workspace=r["ws"])
        prefix_attention(kv, q, go, pre, **args)
        torch.cuda.synchronize()
        with torch.cuda.graph(r["graph"], stream=r["stream"]):
            prefix_attention(kv, q, go, pre, **args)
        runs.append(r)
    for lens in ([200, 170, 900], [1, 16, 0], [33, 0, 129], [0, 0, 0], [200, 1, 17]):
        c.lens = lens
        c.seq_len.copy_(_ints(lens))
        torch.cuda.synchronize()
        for r in runs:
            with torch.cuda.stream(r["stream"]):
                r["graph"].replay()
        torch.cuda.synchronize()
        for r in runs:
            check_attention(c, q, r["out"], r["lse"], [1, 1], [0, 1], [(0, 2, 2)], True, 1 / 8)


def test_bad_entries_are_reported():
    import torch
    from block_diffusion_speculative_hidden_gb300 import _lib, prefix_attention
    from decode_ref import Cache, check_attention
    for what, bit in [("rows", _lib.DEV_BAD_ROWS), ("rows_negative", _lib.DEV_BAD_ROWS), ("seq", _lib.DEV_BAD_BLOCK),
                      ("prefix", _lib.DEV_BAD_BLOCK), ("prefix_negative", _lib.DEV_BAD_BLOCK),
                      ("long", _lib.DEV_SEQ_TOO_LONG), ("long_prefix", _lib.DEV_SEQ_TOO_LONG),
                      ("page", _lib.DEV_BAD_PAGE), ("page_negative", _lib.DEV_BAD_PAGE), ("bounds", _lib.DEV_BAD_BLOCK),
                      ("bounds_first", _lib.DEV_BAD_BLOCK), ("bounds_last", _lib.DEV_BAD_BLOCK)]:
        for T in (2, 17):
            c = Cache([20, 32, 40, 48], 2, 64, torch.bfloat16, 5, max_pages=3)
            n, seq, go, pre = _ints([T, T, T]), _ints([0, 1, 2]), _ints([0, 1, 3]), _ints([-1, 3])
            if what.startswith("rows"):
                n[1] = T + 1 if what == "rows" else -1
            elif what == "seq":
                seq[1] = 4
            elif what.startswith("prefix"):
                pre[1] = 4 if what == "prefix" else -2
            elif what == "long":
                c.seq_len[1] = 1 << 30
                c.table[1] = c.table[3]
            elif what == "long_prefix":
                c.seq_len[3] = 49
            elif what.startswith("page"):
                c.table[1, 1] = c.k.shape[0] if what == "page" else -5
            elif what == "bounds":
                go[1] = 7
            elif what == "bounds_first":
                go[0] = -1
            elif what == "bounds_last":
                go[2] = 4
            q = torch.randn(3, T, 8, 64, device="cuda", dtype=torch.bfloat16)
            out = torch.full((3, T, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros(3, T, 8, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            prefix_attention(c.paged(), q, go, pre, n, seq=seq, out=out, lse=lse, status=status)
            assert int(status.item()) == bit, (what, T)
            assert torch.isfinite(out.float()).all()
            if what.startswith("rows"):
                assert (out[1] == 7.0).all()
            if not what.startswith("bounds"):      # entry 0 has a sound group and sequence of its own
                check_attention(c, q, out, lse, [T, 0, 0], [0, 1, 2], [(0, 3, -1)], True, 1 / 8)
            else:                                  # without sound bounds nobody has a prefix
                check_attention(c, q, out, lse, [T, T, T], [0, 1, 2], [(0, 3, -1)], True, 1 / 8)


def test_drafter_cache_with_a_shared_prefix():
    """Sequences of a drafter's cache behind a prefix injected into one of its sequences."""
    import numpy as np
    import torch
    import synth
    from block_diffusion_speculative_hidden_gb300 import Drafter, prefix_attention, weights_to_device
    from decode_ref import check_attention
    cfg = synth.MINI_CONFIGS["mini_a"].replace(batch=3, n_layers=2)
    dr = Drafter(cfg, weights_to_device(synth.make_weights(cfg), cfg.dtype), max_batch=3, max_pages_per_seq=8,
                 n_pages=24, max_rows=100, max_inject_rows=300)
    lens = [9, 31, 100]
    feats = torch.randn(3, 100, cfg.feat_dim, device="cuda").bfloat16()
    dr.inject_kv(feats, _ints(lens))
    q = torch.randn(2, 3, cfg.n_q_heads, cfg.head_dim, device="cuda", dtype=torch.float16)
    for layer in range(2):
        kv = dr.paged_kv(layer)
        lse = torch.empty(2, 3, cfg.n_q_heads, device="cuda")
        out = prefix_attention(kv, q, _ints([0, 2]), _ints([2]), lse=lse)

        class C:
            k, v = kv.k, kv.v
            table = dr.page_table

            @staticmethod
            def tokens(pool, s):
                i = torch.arange(lens[s], device="cuda")
                return pool[dr.page_table[s].long()[i // 16], :, i % 16].double()
        C.lens = lens
        check_attention(C, q, out, lse, [3, 3], [0, 1], [(0, 2, 2)], True, 1 / math.sqrt(cfg.head_dim))
    assert dr.device_status() == 0
    dr.close()


def test_many_short_sequences():
    """More entries than the CTAs keep in shared memory, several of them a warp; most and fewest that a call takes."""
    lens = [(7 * b) % 41 for b in range(600)]
    _run(600, 1, 4, 1, 64, "float16", lens)
    _run(600, 2, 4, 1, 128, "bfloat16", lens, [(2, (13 * g) % 70) for g in range(300)], n=[b % 3 for b in range(600)])
    _run(4096, 1, 2, 1, 64, "float16", [b % 5 for b in range(4096)], [(2, g % 3 * 9) for g in range(2048)])


def test_short_prefixes_of_few_rows():
    # groups of 8 rows and fewer a kv head: prefixes and own parts on one line of pages
    _run(7, 1, 8, 4, 64, "bfloat16", [5, 0, 17, 300, 33, 1, 64], [(1, 40), (3, 500), (0, 16), (1, None), (2, 129)])
    _run(4, 2, 8, 2, 128, "float16", [2, 18, 90, 5], [(1, 1000), (1, 17), (1, 0), (1, 64)], n=[1, 0, 2, 2])
    # on average: one group has 40 rows
    _run(25, 1, 4, 1, 64, "float16", [3 * b for b in range(25)], [(1, 33)] * 15 + [(10, 250)])


@pytest.mark.parametrize("dtype,dh,Hq,Hkv,B", [("float16", 64, 64, 8, 44), ("bfloat16", 128, 24, 8, 112)])
def test_live_rows_of_a_large_batch(dtype, dh, Hq, Hkv, B):
    """Row tiles that hold live rows of several entries, some of them without any."""
    n = [(5 * b + 3) % 17 for b in range(B)]
    lens = [(37 * b) % 90 for b in range(B)]
    for rows in (n, [16] * B, [0] * 9 + [1] * (B - 9)):
        _run(B, 16, Hq, Hkv, dh, dtype, lens, [(9, 260), (0, 70), (3, None), (B - 13, 700), (1, 31)], n=rows)
    _run(B, 16, Hq, Hkv, dh, dtype, lens, [(B, 150)], n=n, causal=False, in_place=False)


@pytest.mark.parametrize("T", [1, 17])
def test_nan_stays_in_its_rows(T):
    """A NaN query gives NaN in its row and in no other; a NaN key that no row sees gives none."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache, check_attention
    for dh in (64, 128):
        c = Cache([T + 40, T, 500], 2, dh, torch.float16, 9)
        q = torch.randn(2, T, 8, dh, device="cuda", dtype=torch.float16)
        want, lw = torch.empty_like(q), torch.empty(2, T, 8, device="cuda")
        prefix_attention(c.paged(), q, _ints([0, 2]), _ints([2]), out=want, lse=lw)
        check_attention(c, q, want, lw, [T, T], [0, 1], [(0, 2, 2)], True, 1 / math.sqrt(dh))
        bad = q.clone()
        bad[1, T - 1, 3, 5] = math.nan
        out, lse = torch.empty_like(q), torch.empty(2, T, 8, device="cuda")
        prefix_attention(c.paged(), bad, _ints([0, 2]), _ints([2]), out=out, lse=lse)
        assert out[1, T - 1, 3].isnan().all() and lse[1, T - 1, 3].isnan()
        out[1, T - 1, 3], lse[1, T - 1, 3] = want[1, T - 1, 3], lw[1, T - 1, 3]
        check_attention(c, q, out, lse, [T, T], [0, 1], [(0, 2, 2)], True, 1 / math.sqrt(dh))
        if T > 1:                                # the last token's key: rows before it do not see it
            page, slot = c.table[0].long()[(T + 39) // 16], (T + 39) % 16
            c.k[page, :, slot] = math.nan
            prefix_attention(c.paged(), q, _ints([0, 2]), _ints([2]), out=out, lse=lse)
            assert out[0, T - 1].isnan().all() and torch.isfinite(out[0, :T - 1].float()).all()
            assert torch.isfinite(out[1].float()).all()


@pytest.mark.parametrize("B,Hkv,own,P", [(2, 2, 700, None), (8, 8, 700, None), (16, 8, 2000, None), (4, 8, 1500, 600),
                                         (16, 8, 900, 900)])
@pytest.mark.parametrize("dh", [64, 128])
def test_own_parts_in_chunks(B, Hkv, own, P, dh):
    """Blocks whose own sequences are long enough to be split, joined afterwards."""
    _run(B, 17, 4 * Hkv, Hkv, dh, "float16", [own - 37 * b for b in range(B)], [(B, P)] if P else [])


@pytest.mark.parametrize("P", [0, 200])
def test_more_than_32_bits_of_rows(P):
    """B T Hq head_dim past 2^31: the last entries of a batch whose other ones have no rows."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache, check_attention
    B, T, Hq, dh = 4096, 65, 64, 128
    assert B * T * Hq * dh > 1 << 31
    c = Cache([70, 90, 0, 200], 8, dh, torch.bfloat16, 3)
    q = torch.zeros(B, T, Hq, dh, device="cuda", dtype=torch.bfloat16)
    q[-2:] = torch.randn(2, T, Hq, dh, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(B, T, Hq, device="cuda")
    n, seq = [0] * (B - 2) + [T, 3], [2] * (B - 2) + [0, 1]
    groups = dict(group_off=_ints([0, B]), prefix_seq=_ints([3]), max_prefix=P) if P else {}
    prefix_attention(c.paged(), q, n_rows=_ints(n), seq=_ints(seq), max_len=90, out=out, lse=lse, **groups)
    check_attention(c, q, out, lse, n, seq, [(0, B, 3)] if P else [], True, 1 / math.sqrt(dh))
