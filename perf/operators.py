"""The decode-step operators around the paged KV cache, as measured cases.

Three operators that a serving step chains: keys and values (and the step's
queries) are rotated and appended to a paged cache; the step's queries attend
to a prefix that a group of sequences shares and to each sequence's own keys;
the projections around them take 4-bit weights with group scales.

`own = False` computes each operator in its plain form (elementary torch
operations in fp32); `own = True` calls the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
PAGE = 16


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one conversation: a call's fixed cost
        dict(name="append one token", op="append", B=1, T=1, Hq=32, Hkv=8, dh=128, src="bf16", kv="bf16",
             n_lo=1, n_hi=1, len_lo=2048, len_hi=2048, base=0, seqs=1),
        # a verified block of up to 17 tokens in each of 128 sequences, straight
        # from an fp32 projection output, behind a shared prompt
        dict(name="append verified blocks", op="append", B=128, T=17, Hq=64, Hkv=8, dh=64, src="f32", kv="f16",
             n_lo=1, n_hi=17, len_lo=300, len_hi=1100, base=1024, seqs=160),
        # prompts of uneven length, keys and values only
        dict(name="append prompts", op="append", B=8, T=4096, Hq=0, Hkv=8, dh=128, src="bf16", kv="f16",
             n_lo=1000, n_hi=4096, len_lo=4096, len_hi=4500, base=0, seqs=8),
        # one conversation behind a short prompt, token by token
        dict(name="decode one sequence", op="attend", B=1, T=1, Hq=32, Hkv=8, dh=128, kv="bf16", NG=1,
             p_lo=500, p_hi=500, len_lo=77, len_hi=77, n_lo=1, n_hi=1, causal=True, orphan=False),
        # a serving batch behind one system prompt, token by token
        dict(name="decode batch", op="attend", B=64, T=1, Hq=32, Hkv=8, dh=128, kv="bf16", NG=1,
             p_lo=8192, p_hi=8192, len_lo=30, len_hi=1500, n_lo=1, n_hi=1, causal=True, orphan=False),
        # the target's check of a drafted block: 17 positions a sequence at once
        dict(name="verify batch", op="attend", B=32, T=17, Hq=32, Hkv=8, dh=128, kv="f16", NG=1,
             p_lo=8190, p_hi=8190, len_lo=17, len_hi=700, n_lo=17, n_hi=17, causal=True, orphan=False),
        # several questions about one long document
        dict(name="decode long document", op="attend", B=4, T=1, Hq=32, Hkv=8, dh=128, kv="f16", NG=1,
             p_lo=131000, p_hi=131000, len_lo=1, len_hi=300, n_lo=1, n_hi=1, causal=True, orphan=False),
        # blocks whose positions see each other, several prompts, sequences
        # without one, uneven block lengths, sequences with nothing of their own
        dict(name="draft blocks in groups", op="attend", B=48, T=16, Hq=64, Hkv=8, dh=64, kv="f16", NG=5,
             p_lo=40, p_hi=5000, len_lo=0, len_hi=600, n_lo=1, n_hi=16, causal=False, orphan=True),
        # q, k and v of one token
        dict(name="w4 qkv of one token", op="w4", M=1, N=6144, K=4096, group=128, fmt="int4", zero=False, x="bf16",
             scale="bf16"),
        # gate and up rows for a block of 16
        dict(name="w4 gate up of a block", op="w4", M=16, N=24576, K=4096, group=64, fmt="int4", zero=True, x="f16",
             scale="f16"),
        # the vocabulary's rows for one token
        dict(name="w4 vocabulary of one token", op="w4", M=1, N=151936, K=4096, group=32, fmt="e2m1", zero=False,
             x="bf16", scale="bf16"),
        # 17 positions to check, a width that fills no tile
        dict(name="w4 narrow verify", op="w4", M=17, N=2880, K=2880, group=32, fmt="int4", zero=True, x="bf16",
             scale="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "w4"])
    if op == "w4":
        group = rng.choice([32, 64, 128])
        K = 32 * _log(rng, 2, 384)
        N = _log(rng, 16, 152000)
        M = rng.choice([1, 1, _log(rng, 1, 32)])
        while N * K > 151936 * 4096 or M * N > 1500000:
            N = N // 2 + 1
        fmt = rng.choice(["int4", "int4", "e2m1"])
        return dict(op=op, M=M, N=N, K=K, group=group, fmt=fmt, zero=fmt == "int4" and rng.random() < 0.5,
                    x=rng.choice(["bf16", "f16"]), scale=rng.choice(["bf16", "f16", "f32"]))
    dh = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    if op == "append":
        B, T = _log(rng, 1, 160), _log(rng, 1, 3000)
        while B * T > 20000:
            B = B // 2 + 1
            T = T // 2 + 1
        kv = rng.choice(["bf16", "f16", "f32"])
        hi = T + _log(rng, 1, 1000)
        return dict(op=op, B=B, T=T, Hq=rng.choice([0, G * Hkv]), Hkv=Hkv, dh=dh,
                    src="f32" if kv == "f32" else rng.choice(["bf16", "f16", "f32"]), kv=kv,
                    n_lo=max(1, T // 3), n_hi=T, len_lo=T, len_hi=hi, base=rng.choice([0, _log(rng, 1, 30000)]),
                    seqs=B + rng.randrange(5))
    B, T = _log(rng, 1, 128), rng.choice([1, 1, 2, 5, 8, 16, 17])
    NG = min(B, rng.choice([1, 1, 2, 3, 6]))
    p_hi = _log(rng, 16, 131000)
    while B * T * G * Hkv * p_hi * dh > 32 * 17 * 32 * 8190 * 128 // 2 or NG * p_hi > 131000:
        p_hi = p_hi // 2 + 1
        B = max(NG, B - B // 8)
    len_hi = T + _log(rng, 1, 2000)
    return dict(op=op, B=B, T=T, Hq=G * Hkv, Hkv=Hkv, dh=dh, kv=rng.choice(["bf16", "f16"]), NG=NG,
                p_lo=p_hi // rng.choice([1, 2, 5]) + 1, p_hi=p_hi + 1, len_lo=rng.choice([0, T]), len_hi=len_hi,
                n_lo=rng.choice([1, T]), n_hi=T, causal=rng.random() < 0.75, orphan=NG > 1 and rng.random() < 0.5)


def _spread(lo, hi, n, shift=1):
    """n whole numbers spread over lo .. hi, the same ones every time."""
    return [lo + int((hi - lo + 1) * (((i + shift) * 0.6180339887498949) % 1.0)) for i in range(n)]


def _shape(c):
    """Lengths of a cache case: new rows and length of every sequence; for attend also group bounds and prefix lengths."""
    n = _spread(c["n_lo"], c["n_hi"], c["B"], 2)
    lens = _spread(c["len_lo"], c["len_hi"], c["B"], 1)
    if c["op"] == "append":
        return n, lens
    cuts = sorted(_spread(1, c["B"] - 1, c["NG"] - 1, 3)) if c["NG"] > 1 else []
    pre = _spread(c["p_lo"], c["p_hi"], c["NG"], 4)
    if c["orphan"]:
        pre[-1] = 0
    return n, lens, [0] + cuts + [c["B"]], pre


def _visible(c):
    """(query rows, (row, key) pairs that are attended) of an attend case, for one query head."""
    n, lens, off, pre = _shape(c)
    rows = pairs = 0
    for g in range(c["NG"]):
        for b in range(off[g], off[g + 1]):
            rows += n[b]
            for t in range(n[b]):
                pairs += pre[g] + (max(0, lens[b] - n[b] + t + 1) if c["causal"] else lens[b])
    return rows, pairs


def work(c):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] == "w4":
        groups = -(-c["K"] // c["group"])
        w = c["N"] * c["K"] // 2 + c["N"] * groups * (size[c["scale"]] + (1 if c["zero"] else 0))
        return {"bytes": w + c["M"] * c["K"] * 2 + c["M"] * c["N"] * 4, "flops": 2 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "append":
        n, _ = _shape(c)
        rows = sum(n)
        moved = rows * c["dh"] * (2 * c["Hkv"] + c["Hq"]) * (size[c["src"]] + size[c["kv"]])
        return {"bytes": moved + rows * c["dh"] * 4, "flops": rows * c["dh"] * (c["Hkv"] + c["Hq"]) * 3}
    n, lens, off, pre = _shape(c)
    rows, pairs = _visible(c)
    kv = (sum(lens) + sum(pre)) * 2 * c["Hkv"] * c["dh"] * 2
    return {"bytes": kv + rows * c["Hq"] * (c["dh"] * 4 + 4), "flops": 4 * pairs * c["Hq"] * c["dh"]}


# ------------------------------------------------------------------ the inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, mul=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * mul).to(dtype)

    s = {"case": c}
    if c["op"] == "w4":
        groups = -(-c["K"] // c["group"])
        s["W"] = torch.randint(0, 256, (c["N"], c["K"] // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scale"] = (torch.rand(c["N"], groups, generator=g, device="cuda") * 0.01 + 0.002).to(DTYPES[c["scale"]])
        s["zero"] = (torch.randint(4, 13, (c["N"], groups), generator=g, device="cuda", dtype=torch.uint8)
                     if c["zero"] else None)
        s["X"] = normal(c["M"], c["K"], dtype=DTYPES[c["x"]])
        return s

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    kvt, B, T, Hkv, dh = DTYPES[c["kv"]], c["B"], c["T"], c["Hkv"], c["dh"]
    if c["op"] == "append":
        n, lens = _shape(c)
        rows = c["seqs"]
        all_len = [0] * rows
        where = torch.randperm(rows, generator=torch.Generator().manual_seed(seed))[:B].tolist()
        for b, r in enumerate(where):
            all_len[r] = lens[b]
        src = DTYPES[c["src"]]
        # one projection's output: every token's q, k and v side by side
        heads = c["Hq"] + 2 * Hkv
        qkv = normal(B, T, heads, dh, dtype=src)
        s["q"] = qkv[:, :, :c["Hq"]] if c["Hq"] else None
        s["k"], s["v"] = qkv[:, :, c["Hq"]:c["Hq"] + Hkv], qkv[:, :, c["Hq"] + Hkv:]
        s["q_out"] = torch.zeros(B, T, c["Hq"], dh, dtype=kvt, device="cuda") if c["Hq"] else None
        s["seq"], s["n_rows"] = ints(where), ints(n)
        s["pos_base"] = torch.full((B,), c["base"], dtype=torch.int32, device="cuda")
        top = c["base"] + max(lens) + 1
        ang = (torch.arange(top, device="cuda", dtype=torch.float64)[:, None]
               * 1.0e6 ** (-torch.arange(dh // 2, device="cuda", dtype=torch.float64) * 2 / dh)[None])
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    else:
        n, lens, off, pre = _shape(c)
        all_len = lens + pre
        rows = len(all_len)
        s["q"] = normal(B, T, c["Hq"], dh, dtype=kvt, mul=2.0)
        s["out"] = torch.zeros(B, T, c["Hq"], dh, dtype=kvt, device="cuda")
        s["lse"] = torch.zeros(B, T, c["Hq"], device="cuda")
        s["n_rows"] = ints(n)
        s["group_off"] = ints(off)
        s["prefix_seq"] = ints([B + i if pre[i] else -1 for i in range(c["NG"])])
        s["max_prefix"], s["max_len"] = max(pre), max(lens)
        s["most"] = max(off[i + 1] - off[i] for i in range(c["NG"]))
    pages = [-(-v // PAGE) for v in all_len]
    ids = torch.randperm(sum(pages) + 3, generator=g, device="cuda").int()
    table = torch.full((rows, max(1, max(pages))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = ids[at:at + p]
        at += p
    s["table"], s["seq_len"] = table, ints(all_len)
    s["kp"] = normal(sum(pages) + 3, Hkv, PAGE, dh, dtype=kvt)
    s["vp"] = normal(sum(pages) + 3, Hkv, PAGE, dh, dtype=kvt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "w4": _own_w4}[op](s)
    return {"append": _plain_append, "attend": _plain_attend, "w4": _plain_w4}[op](s)


def _own_append(s):
    from block_diffusion_speculative_hidden_gb300 import PagedKV, append_kv
    kv = PagedKV(s["kp"], s["vp"], s["table"], s["seq_len"])
    append_kv(kv, s["k"], s["v"], n_rows=s["n_rows"], seq=s["seq"], pos_base=s["pos_base"], rope=(s["cos"], s["sin"]),
              q=s["q"], q_out=s["q_out"])
    return {"k": s["kp"], "v": s["vp"], "q": s["q_out"]}


def _own_attend(s):
    from block_diffusion_speculative_hidden_gb300 import PagedKV, prefix_attention
    kv = PagedKV(s["kp"], s["vp"], s["table"], s["seq_len"])
    prefix_attention(kv, s["q"], s["group_off"], s["prefix_seq"], n_rows=s["n_rows"], causal=s["case"]["causal"],
                     max_prefix=s["max_prefix"], max_len=s["max_len"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_w4(s):
    from block_diffusion_speculative_hidden_gb300 import gemm_w4
    return gemm_w4(s["W"], s["scale"], s["X"], zero=s["zero"], group=s["case"]["group"], fmt=s["case"]["fmt"])


def _plain_append(s):
    B, T = s["k"].shape[:2]
    # the rows behind a sequence's last new one repeat that one
    n = s["n_rows"].long()
    t = torch.minimum(torch.arange(T, device="cuda")[None, :], n[:, None] - 1)
    slot = s["seq_len"][s["seq"].long()].long()[:, None] - n[:, None] + t
    b = torch.arange(B, device="cuda")[:, None]
    pos = s["pos_base"].long()[:, None] + slot
    cos, sin = s["cos"][pos][:, :, None], s["sin"][pos][:, :, None]

    def turned(x):
        x = x[b, t].float()
        half = x.shape[-1] // 2
        x1, x2 = x[..., :half], x[..., half:]
        return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)

    page, at = s["table"][s["seq"].long()[:, None], slot // PAGE].long(), slot % PAGE
    s["kp"][page, :, at] = turned(s["k"]).to(s["kp"].dtype)
    s["vp"][page, :, at] = s["v"][b, t].to(s["vp"].dtype)
    if s["q"] is not None:
        s["q_out"][b, t] = turned(s["q"]).to(s["q_out"].dtype)
    return {"k": s["kp"], "v": s["vp"], "q": s["q_out"]}


def _plain_attend(s):
    q, table = s["q"].float(), s["table"].long()
    B, T, Hq, dh = q.shape
    Hkv, NG, most = s["kp"].shape[1], s["prefix_seq"].shape[0], s["most"]
    G = Hq // Hkv
    off = s["group_off"].long()
    row = s["prefix_seq"].long()
    plen = torch.where(row >= 0, s["seq_len"].long()[row.clamp(min=0)], 0)
    slots = (off[:-1, None] + torch.arange(most, device="cuda")[None]).clamp(max=B - 1)       # [NG, most]
    gid = (torch.arange(B, device="cuda")[:, None] >= off[None, 1:]).sum(1)                   # [B]
    place = torch.arange(B, device="cuda") - off[gid]

    def rows_of(pool, r, longest):
        ids = table[r, :-(-longest // PAGE)].clamp(min=0)
        x = pool[ids].permute(0, 2, 1, 3, 4)
        return x.reshape(x.shape[0], x.shape[1], -1, dh)[:, :, :longest].float()              # [n, Hkv, longest, dh]

    pk = rows_of(s["kp"], row.clamp(min=0), s["max_prefix"])
    pv = rows_of(s["vp"], row.clamp(min=0), s["max_prefix"])
    ok = rows_of(s["kp"], torch.arange(B, device="cuda"), s["max_len"])
    ov = rows_of(s["vp"], torch.arange(B, device="cuda"), s["max_len"])
    qh = q.reshape(B, T, Hkv, G, dh).permute(0, 2, 1, 3, 4)                                    # [B, Hkv, T, G, dh]

    def to_groups(x):                                                                         # [B, Hkv, T, G, d]
        return x[slots].transpose(1, 2).reshape(NG, Hkv, most * T * G, x.shape[-1])

    def to_batch(x):
        return x.reshape(NG, Hkv, most, T, G, x.shape[-1]).transpose(1, 2)[gid, place]

    scale = 1.0 / math.sqrt(dh)
    P, L = pk.shape[2], ok.shape[2]
    sp = to_groups(qh) @ pk.transpose(2, 3) * scale
    sp = to_batch(sp.masked_fill(torch.arange(P, device="cuda") >= plen[:, None, None, None], -math.inf))
    so = (qh.reshape(B, Hkv, T * G, dh) @ ok.transpose(2, 3) * scale).reshape(B, Hkv, T, G, L)
    lens, n = s["seq_len"][:B].long(), s["n_rows"].long()
    t = torch.arange(T, device="cuda")
    seen = (lens - n)[:, None] + t[None] + 1 if s["case"]["causal"] else lens[:, None].expand(B, T)
    so = so.masked_fill(torch.arange(L, device="cuda") >= seen[:, None, :, None, None], -math.inf)
    top = torch.cat([sp, so], -1).amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    ep, eo = torch.exp(sp - top), torch.exp(so - top)
    total = ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True)
    o = to_batch(to_groups(ep) @ pv) + (eo.reshape(B, Hkv, T * G, L) @ ov).reshape(B, Hkv, T, G, dh)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, dh)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hq)
    live = (t[None] < n[:, None])[:, :, None]
    return {"out": torch.where(live[..., None], o, 0.0).to(s["out"].dtype), "lse": torch.where(live, lse, 0.0)}


def _plain_w4(s):
    c, W = s["case"], s["W"]
    codes = torch.stack([W & 15, W >> 4], -1).reshape(W.shape[0], -1)
    if c["fmt"] == "e2m1":
        w = torch.tensor(E2M1, device="cuda")[codes.int()]
    elif s["zero"] is None:
        w = codes.float() - 8.0
    else:
        w = codes.float() - s["zero"].float().repeat_interleave(c["group"], 1)[:, :c["K"]]
    w = w * s["scale"].float().repeat_interleave(c["group"], 1)[:, :c["K"]]
    return s["X"].float() @ w.t()


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "w4":
        table = list(E2M1) if c["fmt"] == "e2m1" else [float(v) for v in range(16)]
        table = torch.tensor(table, dtype=torch.float64, device="cuda")
        out = torch.empty(c["M"], c["N"], dtype=torch.float64, device="cuda")
        k = torch.arange(c["K"], device="cuda")
        for n0 in range(0, c["N"], 8192):
            W = s["W"][n0:n0 + 8192]
            code = (W[:, k // 2].int() >> (4 * (k % 2))[None].int()) & 15
            w = table[code.long()]
            if c["fmt"] == "int4":
                w -= 8.0 if s["zero"] is None else s["zero"][n0:n0 + 8192].double()[:, k // c["group"]]
            w *= s["scale"][n0:n0 + 8192].double()[:, k // c["group"]]
            out[:, n0:n0 + 8192] = s["X"].double() @ w.t()
        return out
    if c["op"] == "append":
        n, lens = _shape(c)
        kp, vp = s["kp"].double(), s["vp"].double()
        qo = s["q_out"].double() if c["Hq"] else None
        half = c["dh"] // 2
        for b in range(c["B"]):
            r = int(s["seq"][b])
            slot = torch.arange(lens[b] - n[b], lens[b], device="cuda")
            cos = s["cos"][c["base"] + slot].double()[:, None]
            sin = s["sin"][c["base"] + slot].double()[:, None]
            at = (s["table"][r].long()[slot // PAGE], slice(None), slot % PAGE)
            x = s["k"][b, :n[b]].double()
            kp[at] = torch.cat([x[..., :half] * cos - x[..., half:] * sin,
                                x[..., half:] * cos + x[..., :half] * sin], -1)
            vp[at] = s["v"][b, :n[b]].double()
            if qo is not None:
                x = s["q"][b, :n[b]].double()
                qo[b, :n[b]] = torch.cat([x[..., :half] * cos - x[..., half:] * sin,
                                          x[..., half:] * cos + x[..., :half] * sin], -1)
        return {"k": kp, "v": vp, "q": qo}
    n, lens, off, pre = _shape(c)
    if _visible(c)[1] * c["Hq"] * c["dh"] * 4 > 4e12:
        return None
    out = torch.zeros(c["B"], c["T"], c["Hq"], c["dh"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["B"], c["T"], c["Hq"], dtype=torch.float64, device="cuda")

    def keys(pool, r, count):
        p = torch.arange(count, device="cuda")
        return pool[s["table"][r].long()[p // PAGE], :, p % PAGE].double().transpose(0, 1)    # [Hkv, count, dh]

    G = c["Hq"] // c["Hkv"]
    for g in range(c["NG"]):
        for b in range(off[g], off[g + 1]):
            k = torch.cat([keys(s["kp"], c["B"] + g, pre[g]), keys(s["kp"], b, lens[b])], 1)
            v = torch.cat([keys(s["vp"], c["B"] + g, pre[g]), keys(s["vp"], b, lens[b])], 1)
            if k.shape[1] == 0:
                lse[b, :n[b]] = -math.inf
                continue
            q = s["q"][b, :n[b]].double().reshape(n[b], c["Hkv"], G, c["dh"]).permute(1, 2, 0, 3)  # [Hkv, G, n, dh]
            z = torch.einsum("hgtd,hkd->hgtk", q, k) / math.sqrt(c["dh"])
            if c["causal"]:
                last = pre[g] + lens[b] - n[b] + torch.arange(n[b], device="cuda")
                z = torch.where(torch.arange(k.shape[1], device="cuda")[None] <= last[:, None], z, -math.inf)
            zl = torch.logsumexp(z, -1)
            p = torch.where(zl[..., None] == -math.inf, 0.0, torch.exp(z - zl[..., None]))
            out[b, :n[b]] = torch.einsum("hgtk,hkd->thgd", p, v).reshape(n[b], c["Hq"], c["dh"])
            lse[b, :n[b]] = zl.permute(2, 0, 1).reshape(n[b], c["Hq"])
    return {"out": out, "lse": lse}
