"""Block tables whose rows map up to 2^31 keys and more, most of them unused: the results of a table that ends with
the sequence, to the bit, or a refusal."""
import numpy as np
import pytest

import forget_ref as R
from test_gpu_evict import dev, table_of
from test_gpu_step_accum import bf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [(1 << 27) - 1, 1 << 27])
def test_calls_on_a_wide_table(pages):
    import torch
    import int8_kv_cache_quant_gb300 as kvq
    kvq.lib()
    kvq.kvq_device_status()
    rng = np.random.default_rng(1)
    n, hkv, G, d, slots = 300, 2, 4, 128, 320
    small, nb = table_of(rng, [n])
    pool = R.Pool.random(rng, nb, hkv, d)
    wide = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    wide[0, :small.shape[1]] = dev(small[0])
    q, q3, k, v = bf(rng, 1, hkv * G, d)[1], bf(rng, 1, 3, hkv * G, d)[1], bf(rng, 1, hkv, d)[1], bf(rng, 1, hkv, d)[1]
    ctx, pos = dev(np.array([n], np.int32)), dev(np.array([n - 1], np.int32))
    res = []
    for table in (dev(small), wide):
        cache, out = pool.to_gpu(kvq), []
        acc = torch.ones((1, hkv, slots), device="cuda")
        sp = torch.arange(slots, dtype=torch.int32, device="cuda").repeat(1, hkv, 1)
        decode = [lambda: kvq.kvq_attn_decode_int8kv(cache, q, table, ctx, slots, 0.1, force_route=1),
                  lambda: kvq.kvq_attn_decode_int8kv(cache, q, table, ctx, slots, 0.1, force_route=2),
                  lambda: kvq.kvq_attn_verify_int8kv(cache, q3, table, ctx, slots, 0.1),
                  lambda: kvq.kvq_decode_step_accum_int8kv(cache, k, v, q, table, ctx, slots, 0.1, acc, slot_pos=sp, pos=pos),
                  lambda: kvq.kvq_decode_step_int8kv(cache, k, v, q, table, ctx, slots, 0.1)]
        for call in decode:
            if pages < 1 << 27:
                out.append(call())
            elif table is wide:
                with pytest.raises(kvq.KvqError) as e:
                    call()
                assert e.value.status == 2
        lens = kvq.kvq_cache_evict(cache, table, ctx, slots, 200, acc, sp, n_sink=4, n_recent=16)[2]
        res.append(out + [acc, sp, lens, cache.k, cache.v, cache.k_scale, cache.v_scale])
    assert kvq.kvq_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*res))
