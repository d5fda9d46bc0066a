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
