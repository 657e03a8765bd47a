"""dflash_append_kv against the rotation in 64 bits: types of source and cache,
strided sources (slices of one projection's rows, unaligned ones), uneven row
counts, positions behind a prefix, slots that end inside a page, a cache past
32-bit offsets, and what must not be touched."""
import numpy as np
import pytest

import synth
from oracle import dflash_oracle as O

pytestmark = pytest.mark.gpu

F32, BF16, F16 = "float32", "bfloat16", "float16"


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(B, T, Hq, Hkv, dh, src, dst, lens, n, base=None, seq=None, rope=True, ld_pad=0, seed=1, **kw):
    """One call and its checks; lens: length of every cache sequence after the append."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import append_kv, rope_table
    from decode_ref import Cache, close_rotated, rounding
    src, dst = getattr(torch, src), getattr(torch, dst)
    c = Cache(lens, Hkv, dh, dst, seed, **kw)
    k0, v0 = (c.k.clone(), c.v.clone()) if not kw.get("first_page") else (None, None)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    width = (Hq + 2 * Hkv) * dh + ld_pad
    raw = torch.randn(B * T * width + 8, generator=g, device="cuda").to(src)
    flat = raw[ld_pad:ld_pad + B * T * width].view(B, T, width)
    cut = lambda h0, h1: flat[:, :, h0 * dh:h1 * dh].unflatten(2, (h1 - h0, dh))
    q = cut(0, Hq) if Hq else None
    k, v = cut(Hq, Hq + Hkv), cut(Hq + Hkv, Hq + 2 * Hkv)
    table = rope_table(max(lens) + (max(base) if base else 0) + 1, dh, 1.0e6) if rope else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((B, T, Hq, dh), 7.0, dtype=dst, device="cuda") if Hq else None
    append_kv(c.paged(), k, v, n_rows=None if n is None else _ints(n), seq=None if seq is None else _ints(seq),
              pos_base=None if base is None else _ints(base), rope=table, q=q, q_out=q_out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    written = torch.zeros(c.k.shape[0], 16, dtype=torch.bool, device="cuda") if k0 is not None else None
    for b in range(B):
        s, nb = (seq[b] if seq else b), (n[b] if n else T)
        slot = torch.arange(lens[s] - nb, lens[s], device="cuda")
        page = c.table[s].long()[slot // 16]
        pos = slot + (base[b] if base else 0)
        got_k, got_v = c.k[page, :, slot % 16], c.v[page, :, slot % 16]
        cos = table[0][pos] if rope else torch.ones(nb, dh // 2, device="cuda")
        sin = table[1][pos] if rope else torch.zeros(nb, dh // 2, device="cuda")
        close_rotated(got_k, k[b, :nb], cos, sin)
        assert torch.equal(got_v, v[b, :nb].to(dst))          # one rounding, to nearest even
        if not rope:
            assert torch.equal(got_k, k[b, :nb].to(dst))
        if Hq:
            close_rotated(q_out[b, :nb], q[b, :nb], cos, sin)
            assert (q_out[b, nb:] == 7.0).all()               # rows behind the last one stay
        if written is not None:
            written[page, slot % 16] = True
    if k0 is not None:                                        # every other slot keeps its bits
        keep = ~written[:, None, :, None].expand_as(c.k)
        for old, new in ((k0, c.k), (v0, c.v)):
            bits = torch.int32 if dst == torch.float32 else torch.int16
            assert torch.equal(old.view(bits)[keep], new.view(bits)[keep])


@pytest.mark.parametrize("src", [F32, BF16, F16])
@pytest.mark.parametrize("dst", [F32, BF16, F16])
@pytest.mark.parametrize("dh", [32, 64, 128])
def test_types(src, dst, dh):
    _run(3, 5, 4, 2, dh, src, dst, [5, 40, 17, 0], [5, 1, 3], base=[0, 100, 7])


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 32, 8), (1, 0, 1), (17, 8, 8), (2, 5, 1), (33, 0, 3)])
def test_heads_and_rows(T, Hq, Hkv):
    lens = [T, T + 15, T + 16, 2 * T + 100, T + 1]
    _run(4, T, Hq, Hkv, 128, BF16, F16, lens, None, seq=[4, 0, 3, 2])


def test_uneven_rows_some_empty():
    _run(6, 17, 64, 8, 64, F32, F16, [0, 1, 20, 16, 700, 33], [0, 1, 17, 16, 3, 0], base=[5, 1024, 0, 9, 30000, 1])


def test_without_rotation():
    _run(2, 9, 4, 2, 64, F32, BF16, [9, 100], [9, 4], rope=False)


@pytest.mark.parametrize("src,pad", [(BF16, 1), (F16, 3), (F32, 2), (BF16, 8), (F32, 4)])
def test_rows_that_are_not_16_byte_aligned(src, pad):
    _run(3, 4, 4, 2, 64, src, BF16, [4, 21, 9], [4, 2, 3], ld_pad=pad)


def test_long_prompt():
    _run(2, 3000, 0, 8, 128, BF16, BF16, [3000, 4100], [3000, 2500])


def test_offsets_past_32_bits():
    # pages from 140000 on: 140000 * 8 * 16 * 128 elements > 2^31
    _run(2, 3, 8, 8, 128, BF16, BF16, [40, 3], [3, 3], first_page=140000)


def test_rounding_of_large_values_to_fp16():
    """Past the range of fp16 a value becomes an infinity of its sign, as a rounding to nearest gives."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import append_kv
    from decode_ref import Cache
    c = Cache([1], 1, 64, torch.float16, 3)
    x = torch.full((1, 1, 1, 64), 1e6, device="cuda")
    append_kv(c.paged(), -x, x)
    page = int(c.table[0, 0])
    assert (c.k[page, 0, 0] == -float("inf")).all() and (c.v[page, 0, 0] == float("inf")).all()


def test_table_matches_the_oracle():
    import torch
    from block_diffusion_speculative_hidden_gb300 import rope_table
    cos, sin = rope_table(70000, 128, 1.0e6)
    pos = np.array([0, 1, 2, 999, 4097, 69999])
    c, s = O.rope_cos_sin(pos, 128, 1.0e6)
    at = torch.from_numpy(pos).cuda()
    # fp64 angles up to 7e4 (2^-53 relative: 1e-11 absolute), one rounding to fp32 of a value at most 1
    assert np.abs(cos[at].double().cpu().numpy() - c).max() <= 2.0 ** -24
    assert np.abs(sin[at].double().cpu().numpy() - s).max() <= 2.0 ** -24


def test_bad_entries_are_reported_and_skipped():
    import torch
    from block_diffusion_speculative_hidden_gb300 import _lib, append_kv, rope_table
    from decode_ref import Cache
    cases = [  # (what to break, bit)
        ("rows", _lib.DEV_BAD_ROWS), ("rows_negative", _lib.DEV_BAD_ROWS), ("seq", _lib.DEV_BAD_BLOCK),
        ("seq_negative", _lib.DEV_BAD_BLOCK), ("short", _lib.DEV_BAD_ROWS), ("long", _lib.DEV_SEQ_TOO_LONG),
        ("page", _lib.DEV_BAD_PAGE), ("page_negative", _lib.DEV_BAD_PAGE), ("pos", _lib.DEV_BAD_POS),
        ("pos_negative", _lib.DEV_BAD_POS)]
    for what, bit in cases:
        c = Cache([20, 20], 2, 64, torch.bfloat16, 5)
        n, seq, base = _ints([4, 4]), _ints([0, 1]), _ints([0, 0])
        if what.startswith("rows"):
            n[1] = 5 if what == "rows" else -1
        elif what.startswith("seq"):
            seq[1] = 2 if what == "seq" else -1
        elif what == "short":
            c.seq_len[1] = 3
        elif what == "long":
            c.seq_len[1] = 33
        elif what.startswith("page"):
            c.table[1, 1] = c.k.shape[0] if what == "page" else -1
        elif what.startswith("pos"):
            base[1] = 100 if what == "pos" else -30
        k0 = c.k.clone()
        x = torch.randn(2, 4, 2, 64, device="cuda", dtype=torch.bfloat16)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        append_kv(c.paged(), x, x, n_rows=n, seq=seq, pos_base=base, rope=rope_table(40, 64, 1e4), status=status)
        assert int(status.item()) == bit, what
        # entry 0 is written, nothing else changes
        at = (c.table[0].long()[1], slice(None), slice(0, 4))
        assert torch.isfinite(c.k[at].float()).all() and torch.equal(c.v[at].transpose(0, 1), x[0])
        k0[at] = c.k[at]
        assert torch.equal(k0.view(torch.int16), c.k.view(torch.int16)), what


def test_drafter_cache_grows_and_is_filled():
    """Drafter.extend allocates by the rules of inject_kv; append_kv fills the new slots of every layer."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import Drafter, append_kv, rope_table, weights_to_device
    from decode_ref import close_rotated
    cfg = synth.MINI_CONFIGS["mini_a"].replace(batch=3, n_layers=2)
    dr = Drafter(cfg, weights_to_device(synth.make_weights(cfg), cfg.dtype), max_batch=3, max_pages_per_seq=4,
                 n_pages=6, max_rows=30, max_inject_rows=90)
    rope = rope_table(64, cfg.head_dim, cfg.rope_theta)
    have = np.zeros(3, np.int64)
    g = torch.Generator(device="cuda").manual_seed(9)
    for n in ([17, 0, 3], [2, 16, 30]):
        nr = _ints(n)
        dr.extend(nr)
        have += n
        assert np.array_equal(dr.seq_len.cpu().numpy(), have)
        for layer in range(2):
            k, v = (torch.randn(3, 30, cfg.n_kv_heads, cfg.head_dim, generator=g, device="cuda") for _ in range(2))
            kv = dr.paged_kv(layer)
            append_kv(kv, k, v, n_rows=nr, rope=rope)
            for b in range(3):
                slot = torch.arange(have[b] - n[b], have[b], device="cuda")
                page = dr.page_table[b].long()[slot // 16]
                close_rotated(kv.k[page, :, slot % 16], k[b, :n[b]], rope[0][slot], rope[1][slot])
                assert torch.equal(kv.v[page, :, slot % 16], v[b, :n[b]].half())
    used = dr.page_table[dr.page_table >= 0]
    assert used.numel() == 2 + 1 + 3 and used.unique().numel() == used.numel()
    assert dr.device_status() == 0
    dr.extend(_ints([16, 0, 0]))                      # the pool is empty
    assert dr.device_status() == 1 and np.array_equal(dr.seq_len.cpu().numpy(), have)
    dr.close()


def test_repeated_and_replayed_calls():
    """A recorded append replays with the lengths of the time; another stream; twice the same."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import append_kv, rope_table
    from decode_ref import Cache, close_rotated
    c = Cache([64, 64], 2, 64, torch.bfloat16, 11)
    rope = rope_table(64, 64, 1e4)
    k = torch.randn(2, 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.randn_like(k)
    kv = c.paged()
    c.seq_len.fill_(0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    append_kv_args = dict(rope=rope, stream=stream)
    with torch.cuda.stream(stream):
        c.seq_len.add_(1)
    append_kv(kv, k, v, **append_kv_args)
    graph = torch.cuda.CUDAGraph()
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        c.seq_len.add_(1)
        append_kv(kv, k, v, **append_kv_args)
    for step in range(1, 40):
        new_k, new_v = torch.randn_like(k), torch.randn_like(v)
        k.copy_(new_k)
        v.copy_(new_v)
        graph.replay()
        torch.cuda.synchronize()
        assert c.seq_len.tolist() == [step + 1] * 2
        for b in range(2):
            page = c.table[b].long()[step // 16]
            close_rotated(c.k[page, :, step % 16][None], k[b], rope[0][step:step + 1], rope[1][step:step + 1])
            assert torch.equal(c.v[page, :, step % 16], v[b, 0])
