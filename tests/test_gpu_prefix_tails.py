"""Faint keys beside a dominant one: what an fp16 probability can hold of them,
and single pages of a long context that only some rows look at."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("B,T,own,P", [(1, 1, 40, 0), (2, 1, 700, 33), (4, 1, 20, 900), (3, 17, 50, 0), (3, 17, 40, 300)])
def test_faint_keys_of_fp16_caches(dh, B, T, own, P):
    """Key 0 of a page weighs 1 and carries nothing, the other 15 weigh 2^-26.3 each and carry
    60000: the output is all theirs.  Probabilities enter the second product in fp16, taken
    against 2^-6 of the largest weight at least, so that each is within 2^-11 of itself or
    2^-25 2^-6 of the largest; the output is rounded once.  (Scores: one product of 16-bit
    values, scaled in fp32: 27 2^-22 in the exponent, and 2^-20 for exp2.)"""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache
    low, big = 26.3, 60000.0
    c = Cache([own] * B + [P], 2, dh, torch.float16, 3)
    c.k.zero_()
    c.v.zero_()
    where = (B, min(P, 130)) if P else (0, own)           # the sequence and the token past the page
    for b in ([B] if P else range(B)):
        page = c.table[b].long()[(where[1] - 1) // 16 - 1]
        c.k[page, :, 1:, 0] = -1.0
        c.v[page, :, 1:] = big
        c.k[page, :, 0, 1] = 1.0
    # every other key: so far below that its weight is nothing
    far = torch.ones(c.k.shape[0], dtype=torch.bool, device="cuda")
    for b in ([B] if P else range(B)):
        far[c.table[b].long()[(where[1] - 1) // 16 - 1]] = False
    c.k[far, :, :, 0] = -4.0
    scale = low * math.log(2.0)
    q = torch.zeros(B, T, 8, dh, device="cuda", dtype=torch.float16)
    q[..., 0] = 1.0
    out, lse = torch.empty_like(q), torch.empty(B, T, 8, device="cuda")
    groups = dict(group_off=_ints([0, B]), prefix_seq=_ints([B])) if P else {}
    prefix_attention(c.paged(), q, scale=scale, causal=False, out=out, lse=lse, **groups)
    p = 2.0 ** -low
    ref = 15 * p * big / (1 + 15 * p)
    tol = ref * (2.0 ** -11 * 2 + 27 * 2.0 ** -22 + 2.0 ** -20) + 15 * 2.0 ** -31 * big + 2.0 ** -25
    assert (out.double() - ref).abs().max().item() <= tol, (out.double().min().item(), out.double().max().item(), ref)
    assert (lse.double() - math.log(1 + 15 * p)).abs().max().item() <= 2.0 ** -20
