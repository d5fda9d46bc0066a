"""The rows that the steps take, on the host alone: tensors of the right number of elements in another order are refused."""
import pytest
import torch

import int8_kv_cache_quant_gb300 as k

B, NQ, H, HQ, D = 2, 3, 4, 8, 128


def step(name, q, k_new, v_new, out):
    cache = k.KVCache(4, H, D, device="cpu")
    table, lens = torch.zeros((B, 2), dtype=torch.int32), torch.full((B,), 20, dtype=torch.int32)
    if name == "window":
        return k.kvq_decode_step_window_int8kv(cache, k_new, v_new, q, table, lens, 32, 0.1, 16, out=out)
    return k.kvq_decode_step_accum_int8kv(cache, k_new, v_new, q, table, lens, 32, 0.1, torch.zeros((B, H, 32)), out=out)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("name", ["window", "accum"])
@pytest.mark.parametrize("what,shape", [
    ("k_new", (B, H, NQ, D)), ("v_new", (B, H, NQ, D)), ("k_new", (NQ, B, H, D)), ("v_new", (B, NQ, D, H)), ("k_new", (H, B * NQ, D)),
    ("v_new", (B * H, NQ * D)), ("k_new", (B, NQ, H, D + 1)), ("k_new", (B, NQ, 2 * H, D)), ("out", (B, HQ, NQ, D)), ("out", (NQ, B, HQ, D))])
def test_another_order_is_refused(monkeypatch, name, what, shape):
    monkeypatch.setattr(k.kvq, "_current_device", lambda: -1)  # what tensors of the host say
    args = dict(q=bf(B, NQ, HQ, D), k_new=bf(B, NQ, H, D), v_new=bf(B, NQ, H, D), out=torch.zeros((B, NQ, HQ, D)))
    args[what] = args[what].new_zeros(shape)
    with pytest.raises(ValueError, match=what):
        step(name, **args)


@pytest.mark.parametrize("name", ["window", "accum"])
def test_one_token_of_another_batch_is_refused(monkeypatch, name):
    monkeypatch.setattr(k.kvq, "_current_device", lambda: -1)
    args = dict(q=bf(B, HQ, D), k_new=bf(H, B, D), v_new=bf(B, H, D), out=torch.zeros((B, HQ, D)))
    with pytest.raises(ValueError, match="k_new"):
        step(name, **args)


@pytest.mark.parametrize("shape", [(B, NQ, H, D), (B * NQ, H, D), (B, NQ, H * D), (B * NQ, H * D), (B * NQ * H, D), (B * NQ * H * D,),
                                   (1, B, NQ, H, D), (B, NQ, 1, H, D), (B, 1, NQ, H, 1, D)])
def test_the_same_order_passes(shape):
    t = bf(*shape)
    assert k.kvq._step_rows("f", "x", t, torch.bfloat16, (B, NQ, H, D), -1) == t.data_ptr()


def test_types_and_gaps_are_refused():
    for t in (bf(B, NQ, H, D).float(), bf(B, NQ, H, 2 * D)[..., ::2], bf(B, H, NQ, D).transpose(1, 2)):
        with pytest.raises(ValueError):
            k.kvq._step_rows("f", "x", t, torch.bfloat16, (B, NQ, H, D), -1)
