"""Sizes at the ends of what the calls count, refused on the host before anything is launched."""
import ctypes

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
