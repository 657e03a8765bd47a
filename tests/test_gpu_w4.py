"""dflash_gemm_w4 against the product in 64 bits: formats, zero points, groups
and scale types, one row to 32, widths and depths that fill no tile, and a
decode step that chains it with the paged cache."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _data(M, N, K, group, fmt, zero, x, scale, seed=1):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    gs = -(-K // group)
    W = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sc = (torch.rand(N, gs, generator=g, device="cuda") * 0.02 + 0.001).to(getattr(torch, scale))
    z = torch.randint(0, 16, (N, gs), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    X = torch.randn(M, K, generator=g, device="cuda").to(getattr(torch, x))
    return W, sc, X, z


def _check(M, N, K, group=128, fmt="int4", zero=False, x="bfloat16", scale="bfloat16", seed=1):
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    from decode_ref import check_w4
    W, sc, X, z = _data(M, N, K, group, fmt, zero, x, scale, seed)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M + 1, N), 7.0, device="cuda")
    gemm_w4(W, sc, X, zero=z, group=group, fmt=fmt, out=out[:M], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and (out[M] == 7.0).all()
    check_w4(out[:M], W, sc, X, z, group, fmt)
    return out[:M]


@pytest.mark.parametrize("fmt,zero", [("int4", False), ("int4", True), ("e2m1", False)])
@pytest.mark.parametrize("x", ["bfloat16", "float16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("scale", ["float32", "bfloat16", "float16"])
def test_formats(fmt, zero, x, group, scale):
    _check(1, 80, 512, group, fmt, zero, x, scale)
    _check(9, 45, 288, group, fmt, zero, x, scale)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 24, 25, 31, 32])
def test_rows(M):
    _check(M, 130, 1024, 64, zero=True)
    _check(M, 33, 4096, 32, "e2m1", x="float16")


@pytest.mark.parametrize("N", [1, 15, 16, 17, 31, 33, 127, 129, 1000, 2880, 6144])
@pytest.mark.parametrize("M", [1, 17])
def test_widths(N, M):
    _check(M, N, 2880, 64, zero=True)


@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 256, 288, 1056, 2080, 4096, 8224, 12288])
@pytest.mark.parametrize("M", [1, 16])
def test_depths(K, M):
    _check(M, 50, K, 128, "e2m1")
    _check(M, 50, K, 32, zero=True, x="float16", scale="float32")


def test_wide():
    _check(1, 151936, 512, 64)
    _check(20, 24576, 1024, 128, zero=True)


@pytest.mark.parametrize("M", [1, 8, 16])
def test_many_tiles_and_parts_of_k(M):
    """Several tiles a warp; activations of which shared memory holds a part at a time."""
    _check(M, 24576, 512, 64, zero=True, x="float16", scale="float16")
    _check(M, 40000, 768, 32, "e2m1")
    _check(M, 2500, 12416, 128, zero=True)
    _check(M, 300, 33024, 32, "e2m1", scale="float32")
    _check(M, 48, 16640, 32, zero=True, scale="float32")


def test_scales_and_zero_points_at_any_address():
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    from decode_ref import check_w4
    for group, M in ((32, 1), (64, 9), (128, 16), (128, 17)):
        W, sc, X, z = _data(M, 70, 1024, group, "int4", True, "bfloat16", "float16")
        for shift in (1, 2, 3, 4, 8):
            s2 = torch.zeros(sc.numel() + 8, dtype=sc.dtype, device="cuda")[shift:shift + sc.numel()].view_as(sc)
            z2 = torch.zeros(z.numel() + 8, dtype=z.dtype, device="cuda")[shift:shift + z.numel()].view_as(z)
            s2.copy_(sc)
            z2.copy_(z)
            check_w4(gemm_w4(W, s2, X, zero=z2, group=group), W, sc, X, z, group, "int4")


def test_offsets_past_32_bits():
    """N * K / 2 > 2^31 bytes of codes: the last rows."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    from decode_ref import check_w4
    W, sc, X, z = _data(2, 40000, 131072, 128, "int4", False, "bfloat16", "bfloat16")
    out = gemm_w4(W, sc, X, group=128)
    check_w4(out[:, -48:].contiguous(), W[-48:], sc[-48:], X, None, 128, "int4")


def test_every_code_and_zero_point():
    """Each code times one, exactly: the value table itself; zero points up to 128."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    from decode_ref import w4_values
    for x in (torch.bfloat16, torch.float16):
        for fmt in ("int4", "e2m1"):
            codes = torch.arange(16, dtype=torch.uint8, device="cuda").repeat(2)          # 32 elements
            W = (codes[0::2] | (codes[1::2] << 4))[None].repeat(40, 1).contiguous()
            zero = None
            if fmt == "int4":
                zero = torch.linspace(0, 128, 40, device="cuda").to(torch.uint8)[:, None].contiguous()
            sc = torch.full((40, 1), 0.5, device="cuda")
            for k in range(32):
                X = torch.zeros(1, 32, dtype=x, device="cuda")
                X[0, k] = 1.0
                out = gemm_w4(W, sc, X, zero=zero, group=32, fmt=fmt)
                assert torch.equal(out[0].double(), w4_values(W, sc, zero, 32, fmt)[:, k])


def test_same_on_any_stream_and_when_recorded():
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    W, sc, X, z = _data(17, 300, 2048, 64, "int4", True, "bfloat16", "float16")
    ref = gemm_w4(W, sc, X, zero=z, group=64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = gemm_w4(W, sc, X, zero=z, group=64, stream=s)
    out = torch.zeros_like(ref)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        gemm_w4(W, sc, X, zero=z, group=64, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, other) and torch.equal(ref, out)


@pytest.mark.parametrize("M,K,group,fmt,zero", [(1, 2048, 32, "e2m1", False), (16, 12288, 64, "int4", True),
                                                (24, 2048, 128, "int4", True)])
def test_recordings_at_the_same_time(M, K, group, fmt, zero):
    """Two recordings replayed together over new activations, beside eager calls: the bits of a call by itself."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    W, sc, X, z = _data(M, 700, K, group, fmt, zero, "bfloat16", "bfloat16")
    runs = []
    for _ in range(2):
        r = dict(x=X.clone(), out=torch.zeros(M, 700, device="cuda"), graph=torch.cuda.CUDAGraph(),
                 stream=torch.cuda.Stream())
        gemm_w4(W, sc, r["x"], zero=z, group=group, fmt=fmt, out=r["out"])
        torch.cuda.synchronize()
        with torch.cuda.graph(r["graph"], stream=r["stream"]):
            gemm_w4(W, sc, r["x"], zero=z, group=group, fmt=fmt, out=r["out"])
        runs.append(r)
    for step in range(3):
        xs = [X * (step + 1), X.flip(0) * -1.5]
        want = [gemm_w4(W, sc, x, zero=z, group=group, fmt=fmt) for x in xs]
        for r, x in zip(runs, xs):
            r["x"].copy_(x)
        torch.cuda.synchronize()
        for r in runs:
            with torch.cuda.stream(r["stream"]):
                r["graph"].replay()
        beside = gemm_w4(W, sc, xs[0], zero=z, group=group, fmt=fmt)
        torch.cuda.synchronize()
        assert all(torch.equal(r["out"], w) for r, w in zip(runs, want)) and torch.equal(beside, want[0])


@pytest.mark.parametrize("T,n", [(1, [1, 1, 1]), (17, [17, 3, 9])])
def test_a_decode_step(T, n):
    """q, k, v of a few tokens from 4-bit weights, appended behind a shared prefix, attended to and projected:
    every stage against its definition on the stage before it."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import append_kv, gemm_w4, prefix_attention, rope_table
    from decode_ref import Cache, check_attention, check_w4, close_rotated
    B, Hq, Hkv, dh, d, P = 3, 8, 2, 64, 512, 200
    lens = [n[0] + 30, n[1], n[2] + 1]
    c = Cache(lens + [P], Hkv, dh, torch.bfloat16, 3)
    Wqkv, sq, _, zq = _data(1, (Hq + 2 * Hkv) * dh, d, 64, "int4", True, "bfloat16", "bfloat16", 4)
    Wo, so, _, _ = _data(1, d, Hq * dh, 32, "e2m1", False, "bfloat16", "float32", 5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = rope_table(P + max(lens), dh, 1e6)
    n_rows, base = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (n, [P] * B))
    go, pre = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, B], [B]))
    q = torch.zeros(B, T, Hq, dh, dtype=torch.bfloat16, device="cuda")
    kv = c.paged()
    rows_at_once = 32 // T * T                    # whole entries, at most 32 rows a product
    x = torch.randn(B * T, d, device="cuda").bfloat16()
    qkv = torch.cat([gemm_w4(Wqkv, sq, x[i:i + rows_at_once], zero=zq, group=64, status=status)
                     for i in range(0, B * T, rows_at_once)])
    check_w4(qkv, Wqkv, sq, x, zq, 64, "int4")
    heads = qkv.view(B, T, Hq + 2 * Hkv, dh)
    append_kv(kv, heads[:, :, Hq:Hq + Hkv], heads[:, :, Hq + Hkv:], n_rows, pos_base=base, rope=rope,
              q=heads[:, :, :Hq], q_out=q, status=status)
    for b in range(B):
        slot = torch.arange(lens[b] - n[b], lens[b], device="cuda")
        at = (c.table[b].long()[slot // 16], slice(None), slot % 16)
        close_rotated(c.k[at], heads[b, :n[b], Hq:Hq + Hkv], rope[0][P + slot], rope[1][P + slot])
        close_rotated(q[b, :n[b]], heads[b, :n[b], :Hq], rope[0][P + slot], rope[1][P + slot])
    lse = torch.zeros(B, T, Hq, device="cuda")
    out = torch.zeros(B, T, Hq, dh, dtype=torch.bfloat16, device="cuda")
    prefix_attention(kv, q, go, pre, n_rows, out=out, lse=lse, status=status)
    check_attention(c, q, out, lse, n, [0, 1, 2], [(0, B, B)], True, 1 / math.sqrt(dh))
    a = out.view(B * T, Hq * dh)[:32]
    check_w4(gemm_w4(Wo, so, a, group=32, fmt="e2m1", status=status), Wo, so, a, None, 32, "e2m1")
    assert int(status.item()) == 0
