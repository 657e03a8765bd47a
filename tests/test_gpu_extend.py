"""Drafter.extend (and inject_kv) refuse sequences that the context does not have, whatever the sum overflows to."""
import pytest

import synth

pytestmark = pytest.mark.gpu


def test_sequences_out_of_range_are_refused():
    import torch
    from block_diffusion_speculative_hidden_gb300 import DflashError, Drafter, weights_to_device
    cfg = synth.MINI_CONFIGS["mini_a"].replace(batch=3, n_layers=1)
    dr = Drafter(cfg, weights_to_device(synth.make_weights(cfg), cfg.dtype), max_batch=3, max_pages_per_seq=4,
                 n_pages=6, max_rows=30, max_inject_rows=90)
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    feats = torch.zeros(2, 1, cfg.feat_dim, device="cuda").bfloat16()
    for first in (2, 3, 1 << 20, (1 << 31) - 2, (1 << 31) - 1, -1):
        with pytest.raises(DflashError):
            dr.extend(n, first_seq=first)
        with pytest.raises(DflashError):
            dr.inject_kv(feats, n, first_seq=first)
    dr.extend(n, first_seq=1)
    assert dr.seq_len.tolist() == [0, 1, 1] and dr.device_status() == 0
    dr.close()
