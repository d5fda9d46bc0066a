"""A prompt chunk's result over its own queries, on the host alone: refused."""
import pytest
import torch

import int8_kv_cache_quant_gb300 as k


@pytest.mark.parametrize("shift", [0, 1, 9, -9])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_out_over_q_is_refused(monkeypatch, shift, dtype):
    monkeypatch.setattr(k.kvq, "_current_device", lambda: -1)  # what tensors of the host say
    cache, row = k.KVCache(4, 2, 128, device="cpu"), torch.zeros(4, dtype=torch.int32)
    flat = torch.zeros(64 * 4 * 128, dtype=torch.bfloat16)
    at = 20 * 4 * 128
    q = flat[at:at + 10 * 4 * 128].view(10, 4, 128)
    to = at + shift * 4 * 128
    out = flat[to:to + 10 * 4 * 128 * (2 if dtype is torch.float32 else 1)].view(dtype).view(10, 4, 128)
    with pytest.raises(ValueError, match="overlaps"):
        k.kvq_attn_prefill_window_int8kv(cache, q, 5, row, 0.1, 16, out=out)
