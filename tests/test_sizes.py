"""Sizes at the ends of what the calls count, refused on the host before anything is launched."""
import ctypes

import pytest

import int8_kv_cache_quant_gb300 as k

A = 256  # an aligned address that is never used
UNSUPPORTED = 2


def test_rows_of_a_block_table_that_map_two_to_the_31_keys():
    L, pages = k.lib(), 1 << 27
    c = ctypes.byref(k.kvq._Cache(A, A, A, A, 8, 16, 4, 128))
    ws = 1 << 40
    assert L.kvq_attn_decode_int8kv(c, A, 1, 4, A, pages, A, 100, 0.1, A, A, ws, None, None) == UNSUPPORTED
    assert L.kvq_attn_verify_int8kv(c, A, 1, 2, 4, A, pages, A, 100, 0.1, A, A, ws, None, None) == UNSUPPORTED
    assert L.kvq_decode_step_int8kv(c, A, A, A, 1, 1, 4, A, pages, A, 100, 0.1, A, A, ws, None, None) == UNSUPPORTED
    assert L.kvq_decode_step_accum_int8kv(c, A, A, A, 1, 1, 4, A, pages, A, 100, 0.1, A, A, 100, A, A, A, ws, None,
                                          None) == UNSUPPORTED
    assert L.kvq_debug_stream_floor(c, 1, A, pages, A, 100, 16, None) == UNSUPPORTED


def test_the_automatic_split_takes_contexts_up_to_two_to_the_25():
    for n_sms in (1, 148, 152):
        for d in (128, 256):
            for batch, hkv in ((1, 1), (1, 8), (64, 8), (4000, 16)):
                splits = lambda n: -(-n // k.kvq_decode_auto_split_rows(batch, hkv, d, n, n_sms))  # noqa: E731
                assert max(splits(n) for n in (1 << 25, (1 << 25) - 1, 1 << 24, 1000003)) <= 16384
    assert -(-((1 << 25) + 1) // k.kvq_decode_auto_split_rows(1, 1, 128, (1 << 25) + 1, 152)) == 16385


def test_splits_past_the_bound_are_refused():
    L, c, ws = k.lib(), ctypes.byref(k.kvq._Cache(A, A, A, A, 8, 16, 4, 128)), 1 << 60
    for split, max_ctx in ((16, 16 * 16384 + 1), (2048, (1 << 25) + 1), (65520, (1 << 30))):
        o = ctypes.byref(k.kvq._decode_opts(split, 0, 0))
        assert L.kvq_attn_decode_int8kv(c, A, 1, 4, A, 1 << 26, A, max_ctx, 0.1, A, A, ws, o, None) == UNSUPPORTED
        assert L.kvq_decode_step_accum_int8kv(c, A, A, A, 1, 1, 4, A, 1 << 26, A, max_ctx, 0.1, A, A, max_ctx, A, A, A, ws, o,
                                              None) == UNSUPPORTED


BIG = (1 << 32) + 4  # its low 32 bits are a size that the call would take


@pytest.mark.parametrize("name,args", [
    ("kvq_attn_decode_int8kv", dict(max_ctx=BIG)),
    ("kvq_attn_verify_int8kv", dict(max_ctx=BIG)), ("kvq_decode_step_int8kv", dict(k_new=None, v_new=None, max_ctx=BIG)),
    ("kvq_attn_decode_int8kv_noalloc", dict(max_ctx=BIG, out=None)),
    ("kvq_decode_step_accum_int8kv", dict(k_new=None, v_new=None, max_ctx=BIG, acc=None)),
    ("kvq_debug_stream_floor", dict(max_ctx=BIG)),
    ("kvq_cache_evict", dict(max_ctx=8, keep=BIG)), ("kvq_cache_evict", dict(max_ctx=8, keep=4, n_sink=1 << 32)),
    ("kvq_cache_evict", dict(max_ctx=8, keep=4, n_recent=-(1 << 32))), ("kvq_cache_evict", dict(max_ctx=BIG, keep=4)),
    ("kvq_attn_prefill_int8", dict(history_len=BIG)), ("kvq_attn_prefill_int8_qcodes", dict(history_len=BIG)),
    ("kvq_attn_chunk_weights_int8kv", dict(history_len=1 << 32)),
    ("kvq_rope_bf16", dict(rotary_offset=1 << 32)), ("kvq_rope_bf16", dict(layout=(1 << 32) + 1)),
    ("kvq_rope_quant_write", dict(rotary_dim=BIG)), ("kvq_rope_phases", dict(rotary_dim=BIG))])
def test_numbers_past_32_bits_are_refused(name, args):
    """Before the tensors are looked at: a number that the C call would see cut to its low 32 bits."""
    import inspect
    import torch
    fn = getattr(k, name)
    t = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    need = {n: t for n, p in inspect.signature(fn).parameters.items() if p.default is inspect.Parameter.empty}
    need |= {n: 0.1 for n in need if n == "softmax_scale"} | {n: 16 for n in need if n == "rotary_dim"}
    with pytest.raises(ValueError, match="32 bits"):
        fn(**(need | args))


@pytest.mark.parametrize("call", [
    lambda: k.kvq_evict_workspace_bytes(1, 1, 100, BIG), lambda: k.kvq_chunk_weights_workspace_bytes(BIG, 4, 4, 0, 128),
    lambda: k.kvq_step_accum_workspace_bytes(1, 1, 4, BIG, 128), lambda: k.kvq_decode_workspace_bytes(1, 4, BIG, 128),
    lambda: k.kvq_prefill_workspace_bytes(1, 4, 4, BIG, 128), lambda: k.kvq_sparse_workspace_bytes(BIG, 4, 128),
    lambda: k.kvq_decode_auto_split_rows(1, 4, 128, BIG, 152), lambda: k.kvq_verify_workspace_bytes(1, 1, 4, 100, 128, split_rows=1 << 32)])
def test_sizes_asked_for_past_32_bits_are_refused(call):
    with pytest.raises((ValueError, ctypes.ArgumentError), match="32 bits"):
        call()


@pytest.mark.parametrize("which", [1, 2, 3])
def test_wrapped_tensors_of_different_devices_are_refused(which):
    import torch
    t = [torch.zeros((3, 2, 8, 16, 16), dtype=torch.int8), torch.zeros((3, 2, 128, 16), dtype=torch.int8), torch.zeros((3, 2, 16)),
         torch.zeros((3, 2, 16))]
    assert k.KVCache.wrap(*t).head_dim == 128
    t[which] = t[which].to("meta")
    with pytest.raises(ValueError, match="meta"):
        k.KVCache.wrap(*t)
