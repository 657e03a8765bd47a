"""Every page of a long context, one by one: each query row looks at one page alone, so that a page
that is dropped, read twice, cut short or taken from elsewhere shows as an error of the size of the output."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


CASES = [  # kernels; B, T, Hq, Hkv, context, groups (0: the context is every entry's own sequence), uneven rows
    ("wide prefix", 32, 17, 8, 2, 70001, 1, False),
    ("wide own", 32, 17, 8, 2, 20011, 0, False),
    ("packed prefix", 160, 16, 32, 8, 20011, 1, True),
    ("thin own", 512, 1, 8, 2, 20011, 0, False),
    ("thin prefix", 512, 1, 8, 2, 9009, 256, False),
    ("thin, heads past a tile", 64, 1, 136, 1, 9009, 1, False),
]


@pytest.mark.parametrize("dtype,dh", [("float16", 64), ("bfloat16", 128)])
@pytest.mark.parametrize("what,B,T,Hq,Hkv,L,NG,uneven", CASES)
def test_every_page_alone(dtype, dh, what, B, T, Hq, Hkv, L, NG, uneven):
    """A page's 16 keys are one vector of signs and a row's query is that vector of its page: the page's
    score is above every other's by more than 40 (checked), so the output is the mean of the page's values
    up to 70001 e^-40.  The 16 weights are alike, so that their rounding to the type is one relative error
    of half a step beside the output's; scores are integers and cost 2^-24 of 300 in the exponent."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import PagedKV, prefix_attention
    dt, G, pages = getattr(torch, dtype), Hq // Hkv, -(-L // 16)
    g = torch.Generator(device="cuda").manual_seed(L + dh)
    codes = (torch.randint(0, 2, (pages, Hkv, dh), generator=g, device="cuda") * 2 - 1).to(dt)
    scale = 256.0 / dh
    for h in range(Hkv):
        z = codes[:, h].float() @ codes[:, h].float().t()
        z.fill_diagonal_(-dh)
        assert scale * (dh - z.max().item()) > 40
    order = torch.randperm(pages + 3, generator=g, device="cuda")
    ids = order[:pages]
    k = torch.full((pages + 3, Hkv, 16, dh), math.nan, device="cuda", dtype=dt)
    v = k.clone()
    k[ids] = codes[:, :, None].expand(-1, -1, 16, -1)
    v[ids] = torch.randn(pages, Hkv, 16, dh, generator=g, device="cuda").to(dt)
    if L % 16:
        k[ids[-1], :, L % 16:] = math.nan
        v[ids[-1], :, L % 16:] = math.nan
    held = torch.tensor([16] * (pages - 1) + [L - 16 * (pages - 1)], device="cuda")
    mean = v[ids].double().nan_to_num(0).sum(2) / held[:, None, None]                # [pages, Hkv, dh]
    table = torch.full((2, pages), -1, dtype=torch.int32, device="cuda")
    table[1] = ids.int()
    kv = PagedKV(k, v, table, _ints([0, L]))
    n = [T - b % 3 for b in range(B)] if uneven else [T] * B
    live = torch.tensor(n, device="cuda")[:, None] > torch.arange(T, device="cuda")
    off = [B * i // NG for i in range(NG + 1)] if NG else None
    groups = dict(group_off=_ints(off), prefix_seq=_ints([1] * NG), max_prefix=L, max_len=1) if NG else dict(max_len=L)
    seq = _ints([0 if NG else 1] * B)
    rows = int(live.sum()) * G
    seen = torch.zeros(pages, Hkv, dtype=torch.bool, device="cuda")
    for start in range(0, pages, rows):
        # live rows of every kv head take the pages from `start` on, the last ones first
        at = torch.zeros(B, T, G, dtype=torch.long, device="cuda")
        at[live] = (pages - 1 - start - torch.arange(rows, device="cuda").view(-1, G)) % pages
        q = codes[at].permute(0, 1, 3, 2, 4).reshape(B, T, Hq, dh).contiguous()
        out = torch.empty_like(q)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        prefix_attention(kv, q, n_rows=_ints(n), seq=seq, causal=False, scale=scale, out=out, status=status, **groups)
        assert int(status.item()) == 0
        ref = mean[at].permute(0, 1, 3, 2, 4).reshape(B, T, Hq, dh)
        u = torch.finfo(dt).eps / 2
        err = (out.double() - ref).abs()[live]
        tol = (ref.abs() * (2.02 * u + 300 * 2.0 ** -22 + 2.0 ** -18))[live] + 2.0 ** -24
        assert (err <= tol).all(), (what, (err / tol).max().item())
        seen[at[live].flatten()] = True
    assert seen.all()
