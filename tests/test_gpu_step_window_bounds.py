"""kvq_decode_step_window_int8kv where a bound is far past what a sequence holds: the largest max_ctx and window, and sequences with
fewer keys than rows."""
import numpy as np
import pytest

import forget_ref as R
from test_gpu_evict import dev, table_of
from test_gpu_step_accum import bf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 40, 2 ** 30])
@pytest.mark.parametrize("route", [dict(force_route=1), dict(force_route=2, split_rows=1 << 20)])
@pytest.mark.parametrize("hq,hkv,d,new", [(8, 2, 128, 4), (2, 2, 128, 24), (24, 4, 256, 5)])
def test_fewer_keys_than_rows(kvq, window, route, hq, hkv, d, new):
    """The last rows of such a sequence see its keys, the rows before them none."""
    import torch
    rng = np.random.default_rng(new)
    lens = np.array([1, 300, 0, new - 1, new, 2], np.int32)
    table, nb = table_of(rng, lens)
    pool = R.Pool.random(rng, nb, hkv, d)
    q = bf(rng, len(lens), new, hq, d)[1]
    args = (None, None, q, dev(table), dev(lens))
    got = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), *args, 2 ** 31 - 1, 0.1, window, 4, **route)
    want = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), *args, 304, 0.1, 304, 4, force_route=1)
    assert kvq.kvq_device_status() == 0
    # one split holds all keys: the same sums, and a merge of one part
    assert (got - want).abs().max() <= 2.0 ** -20 * want.abs().max()
    assert bool((want[0, -1] != 0).any()) and bool((got[0, :-1] == 0).all()) and bool((got[2] == 0).all())
