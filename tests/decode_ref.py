"""Inputs of the decode-step operators and their definitions in 64 bits (plain
torch, no kernel of the library)."""
import math

import torch

PAGE = 16


class Cache:
    """A paged cache of random contents: lens[s] tokens in sequence s, pages in
    random order; everything behind a length (and every unused page) is NaN."""

    def __init__(self, lens, Hkv, dh, dtype, seed, spare=3, max_pages=None, device="cuda", first_page=0):
        g = torch.Generator().manual_seed(seed)
        pages = [-(-n // PAGE) for n in lens]
        total = sum(pages) + spare
        self.lens, self.Hkv, self.dh, self.dtype = list(lens), Hkv, dh, dtype
        ids = (torch.randperm(total, generator=g) + first_page).int()
        table = torch.full((len(lens), max_pages or max(1, max(pages))), -1, dtype=torch.int32)
        at = 0
        for s, p in enumerate(pages):
            table[s, :p] = ids[at:at + p]
            at += p
        self.table = table.to(device)
        self.seq_len = torch.tensor(lens, dtype=torch.int32, device=device)
        if first_page:
            self.k = torch.empty((first_page + total, Hkv, PAGE, dh), dtype=dtype, device=device)
            self.v = torch.empty_like(self.k)
            self.k[first_page:] = float("nan")
            self.v[first_page:] = float("nan")
        else:
            self.k = torch.full((total, Hkv, PAGE, dh), float("nan"), dtype=dtype, device=device)
            self.v = self.k.clone()
        gd = torch.Generator(device=device).manual_seed(seed)
        for s, n in enumerate(lens):
            if n:
                i = torch.arange(n, device=device)
                at = (self.table[s].long()[i // PAGE], slice(None), i % PAGE)
                self.k[at] = torch.randn(n, Hkv, dh, generator=gd, device=device).to(dtype)
                self.v[at] = torch.randn(n, Hkv, dh, generator=gd, device=device).to(dtype)

    def paged(self):
        from block_diffusion_speculative_hidden_gb300 import PagedKV
        return PagedKV(self.k, self.v, self.table, self.seq_len)

    def tokens(self, pool, s, n=None):
        """[n, Hkv, dh] fp64: the first n tokens of sequence s."""
        n = self.lens[s] if n is None else n
        i = torch.arange(n, device=pool.device)
        return pool[self.table[s].long()[i // PAGE], :, i % PAGE].double()


def rotate(x, cos, sin):
    """x [n, H, dh] by cos, sin [n, dh / 2], in fp64."""
    h = x.shape[-1] // 2
    c, s = cos.double()[:, None], sin.double()[:, None]
    a, b = x.double()[..., :h], x.double()[..., h:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def rounding(dtype):
    """Half a step of the type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def close_rotated(got, x, cos, sin):
    """got = rotate(x) up to one rounding to got's type and the fp32 pair product: two
    products and a sum, each within 2^-24 of at most |x1| + |x2| (cos, sin at most 1).
    Below the type's normal range its step is tiny * eps."""
    ref = rotate(x, cos, sin)
    h = x.shape[-1] // 2
    mag = (x[..., :h].abs() + x[..., h:].abs()).double()
    tol = rounding(got.dtype) * ref.abs() + 4 * 2.0 ** -24 * torch.cat([mag, mag], -1)
    tol = tol + torch.finfo(got.dtype).tiny * rounding(got.dtype)
    assert ((got.double() - ref).abs() <= tol).all()


def attend_row_block(q, k, v, seen, scale):
    """q [n, Hq, dh] (fp64), k, v [m, Hkv, dh] (fp64), seen [n, m] bool ->
    out [n, Hq, dh], lse [n, Hq], and sum p|v| and the largest |score| error
    weight per row, which the tolerances need."""
    n, Hq, dh = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    z = torch.einsum("nhd,mhd->nhm", q, kk) * scale
    z = torch.where(seen[:, None], z, -math.inf)
    lse = torch.logsumexp(z, -1) if z.shape[-1] else torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.where(lse[..., None] == -math.inf, 0.0, torch.exp(z - lse[..., None])) if z.shape[-1] else z
    out = torch.einsum("nhm,mhd->nhd", p, vv)
    pv = torch.einsum("nhm,mhd->nhd", p, vv.abs())
    zmag = torch.einsum("nhd,mhd->nhm", q.abs(), kk.abs()).amax(-1) * scale if z.shape[-1] else torch.zeros_like(lse)
    return out, lse, pv, zmag


def check_attention(cache, q, out, lse, n, own, groups, causal, scale):
    """out, lse of dflash_prefix_attention against the definition.  own[b]: the
    entry's sequence; groups: [(first, past, prefix sequence or -1)].  Returns
    the number of rows checked.

    Tolerance, with u = rounding(type): a score is an fp32 sum of dh products
    (error at most (dh + 4) 2^-24 times the sum of their magnitudes: `dz`),
    which moves every probability by at most e^(2 dz) - 1 and log-sum-exp by dz;
    the exponentials and the sums over m keys, their partial results and the
    joins add (m + 64) 2^-24 (fp32 additions of same-signed terms) and 2^-20
    (exp2 and log2 on the device); probabilities enter the second product
    rounded to the type (u), below fp16's smallest step 2^-24 by up to 2^-25
    each, against sums of at least 1; the output is rounded once (u)."""
    B, T, Hq, dh = q.shape
    u = rounding(q.dtype)
    rows = 0
    entry_prefix = {b: pre for lo, hi, pre in groups for b in range(lo, hi)}
    for b in range(B):
        nb, s, pre = n[b], own[b], entry_prefix.get(b, -1)
        if nb == 0:
            continue
        L, P = cache.lens[s], cache.lens[pre] if pre >= 0 else 0
        k, v = cache.tokens(cache.k, s), cache.tokens(cache.v, s)
        if P:
            k = torch.cat([cache.tokens(cache.k, pre), k])
            v = torch.cat([cache.tokens(cache.v, pre), v])
        j = torch.arange(P + L, device=q.device)
        i = torch.arange(nb, device=q.device)
        seen = (j[None] < P) | ((j[None] - P) <= (L - nb + i)[:, None] if causal else j[None] >= P)
        ref, rl, pv, zmag = attend_row_block(q[b, :nb].double(), k, v, seen, scale)
        m = P + L
        dz = (dh + 4) * 2.0 ** -24 * zmag
        rel = 2 * dz * 1.01 + (m + 64) * 2.0 ** -24 + 2.0 ** -20 + u
        tol = rel[..., None] * pv + u * ref.abs() * 1.01
        if q.dtype == torch.float16:
            tol = tol + 2.0 ** -25 * m * (v.abs().amax() if m else 0.0) + 2.0 ** -25
        got = out[b, :nb].double()
        assert torch.isfinite(got).all()
        assert ((got - ref).abs() <= tol).all(), (b, ((got - ref).abs() / tol).max().item())
        if lse is not None:
            gl = lse[b, :nb].double()
            dead = rl == -math.inf
            assert torch.equal(gl == -math.inf, dead)
            lt = dz + (m + 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * rl.abs()
            assert ((gl - rl).abs()[~dead] <= lt[~dead]).all()
            assert (got[dead] == 0).all()
        rows += nb
    return rows


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def w4_values(W, scale, zero, group, fmt):
    """The matrix that 4-bit codes and group scales stand for, [N, K] fp64."""
    N, K = W.shape[0], W.shape[1] * 2
    codes = torch.stack([W & 15, W >> 4], -1).reshape(N, K).long()
    if fmt == "e2m1":
        w = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=W.device)[codes]
    else:
        z = torch.full(scale.shape, 8, device=W.device) if zero is None else zero.long()
        w = (codes - z.repeat_interleave(group, 1)[:, :K]).double()
    return w * scale.double().repeat_interleave(group, 1)[:, :K]


def check_w4(out, W, scale, X, zero, group, fmt):
    """Products are exact in fp32; they are added 16 at a time (K / 16 steps), a block's sum
    is scaled and added to the total (K / 32 steps or fewer), and a few partial totals
    are joined.  Every step is within 2^-23 of the magnitudes (the matrix unit's fp32
    additions may truncate), so K / 8 + 16 steps bound them all."""
    w = w4_values(W, scale, zero, group, fmt)
    ref = X.double() @ w.t()
    mag = X.double().abs() @ w.abs().t()
    tol = (W.shape[1] * 2 / 8 + 16) * 2.0 ** -23 * mag
    assert torch.isfinite(out).all()
    assert ((out.double() - ref).abs() <= tol).all(), ((out.double() - ref).abs() / tol.clamp(min=1e-300)).max().item()
