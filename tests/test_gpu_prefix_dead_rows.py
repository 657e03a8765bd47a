"""Rows without a query (i >= n_rows[b], or past a tile's whole tokens) cost the
rows beside them nothing, whatever the caller's buffer holds there."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("Hq", [32, 40])
def test_what_dead_rows_hold_costs_no_time(dh, Hq):
    """The last row of every entry is not one: 32 entries of 16 rows behind 8192 tokens, with zeros, NaN
    or infinities in those rows, take the same time (the least of 30 calls each, taken in turn) and give
    the same bits."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention, prefix_attention_workspace
    from decode_ref import Cache
    B, T, Hkv, P = 32, 17, 8, 8192
    c = Cache([40] * B + [P], Hkv, dh, torch.float16, 3)
    kv = c.paged()
    args = dict(group_off=_ints([0, B]), prefix_seq=_ints([B]), n_rows=_ints([T - 1] * B), max_prefix=P, max_len=40)
    ws = torch.empty(prefix_attention_workspace(kv, Hq, B, T, 1, P, 40), dtype=torch.uint8, device="cuda")
    base = torch.randn(B, T, Hq, dh, device="cuda").half()
    runs = []
    for fill in (0.0, math.nan, math.inf):
        q = base.clone()
        q[:, T - 1:] = fill
        runs.append((q, torch.zeros_like(q), torch.zeros(B, T, Hq, device="cuda"), []))
    for step in range(33):
        for q, out, lse, times in runs:
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda._sleep(200000)              # (the host is ahead: the events time the kernels alone)
            a.record()
            prefix_attention(kv, q, out=out, lse=lse, workspace=ws, **args)
            b.record()
            torch.cuda.synchronize()
            if step >= 3:
                times.append(a.elapsed_time(b))
    clean = min(runs[0][3])
    for q, out, lse, times in runs[1:]:
        assert torch.equal(out, runs[0][1]) and torch.equal(lse, runs[0][2])
        assert min(times) <= 1.2 * clean, (min(times), clean)
