"""Bad prefixes are reported whichever kernel takes the batch, and for groups without entries too."""
import pytest

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind,bit", [("index", 32), ("negative", 32), ("length", 2)])
@pytest.mark.parametrize("size", ["thin", "wide", "packed"])
@pytest.mark.parametrize("where", [0, 1, 70])
def test_bad_prefix_of_an_empty_group(kind, bit, size, where):
    """70 empty groups and one with all entries (the second or the last); one of the empty ones has a bad prefix."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import prefix_attention
    from decode_ref import Cache, check_attention
    B, T, Hkv = {"thin": (2, 1, 2), "wide": (3, 17, 2), "packed": (48, 16, 8)}[size]
    c = Cache([T + b % 5 for b in range(B)] + [64, 20], Hkv, 64, torch.float16, 4)
    full = 1 if where != 1 else 70
    off = [0] * (full + 1) + [B] * (71 - full)
    pre = [B] * 71
    if kind == "length":
        pre[where] = B + 1
        c.seq_len[B + 1] = 16 * c.table.shape[1] + 1
    else:
        pre[where] = B + 2 if kind == "index" else -2
    q = torch.randn(B, T, 8 * Hkv, 64, device="cuda", dtype=torch.float16)
    out, lse = torch.empty_like(q), torch.empty(B, T, 8 * Hkv, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = [T] * B
    prefix_attention(c.paged(), q, _ints(off), _ints(pre), _ints(n), out=out, lse=lse, status=status)
    assert int(status.item()) == bit
    check_attention(c, q, out, lse, n, list(range(B)), [(0, B, B)], True, 1 / 8)
