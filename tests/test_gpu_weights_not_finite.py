"""Attention weights of rows whose scores are not finite: p = 2^(s - M) / l is NaN for every key such a row sees,
wherever the keys are cut into pages, teams, splits, tiles and runs, and nothing for the keys it does not see."""
import numpy as np
import pytest

import forget_ref as R
from test_gpu_chunk_weights import check as check_chunk
from test_gpu_evict import dev, table_of
from test_gpu_step_accum import bf, check as check_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


def set_scale(pool, row, t, h, value):
    """k_scale of key t of KV head h."""
    pool.ks[row[np.asarray(t) // 16], h, np.asarray(t) % 16] = value


@pytest.mark.parametrize("ctx,keys,G,d,nq,split", [
    (17, [16], 1, 128, 1, 0), (17, [16], 4, 256, 1, 0), (17, [0], 2, 256, 1, 16),  # alone in a page, and in a split
    (33, [32], 12, 128, 1, 0), (100, list(range(64, 80)), 6, 256, 1, 32),          # a whole page of NaN
    (130, [129], 3, 256, 4, 128), (65, list(range(64)), 8, 128, 3, 64),            # several rows a sequence; a split of NaN
    (2000, [1999], 4, 128, 1, 64)])
def test_step_with_a_key_of_nan(kvq, ctx, keys, G, d, nq, split):
    rng = np.random.default_rng(ctx + G)
    hkv, lens = 2, [ctx, ctx]
    table, nb = table_of(rng, lens)
    pool = R.Pool.random(rng, nb, hkv, d)
    set_scale(pool, table[0], keys, 1, np.nan)
    q, qt = bf(rng, 2, nq, hkv * G, d)
    acc0 = np.ones((2, hkv, table.shape[1] * 16), np.float32)
    acc = dev(acc0)
    out = kvq.kvq_decode_step_accum_int8kv(pool.to_gpu(kvq), None, None, qt, dev(table), dev(np.array(lens, np.int32)), ctx,
                                           0.07, acc, split_rows=split)
    assert kvq.kvq_device_status() == 0
    a, o = acc.cpu().numpy(), out.cpu().numpy()
    # the last row sees every key, the NaN ones among them
    assert np.isnan(a[0, 1, :ctx]).all() and (a[0, 1, ctx:] == 1).all()
    # the other head, and the other sequence, as ever
    pick = lambda b, h: (table[b:b + 1], [ctx], ctx, q[b:b + 1, :, h * G:(h + 1) * G],  # noqa: E731
                         o[b:b + 1, :, h * G:(h + 1) * G], acc0[b:b + 1, h:h + 1], a[b:b + 1, h:h + 1], 1, 0.07, [False], nq)
    for b, h in ((0, 0), (1, 0), (1, 1)):
        one = R.Pool(*(x[:, h:h + 1] for x in (pool.k, pool.v, pool.ks, pool.vs)))
        check_step(one, *pick(b, h))


@pytest.mark.parametrize("d", [128, 256])
def test_step_whose_new_token_is_infinite(kvq, d):
    """An infinite element makes the row's scale infinite, and the key's score +inf or NaN (every weight of the row is
    NaN) or -inf (the key gets nothing and the others share the row).  It is the first key of a split of its own."""
    rng = np.random.default_rng(3)
    ctx, hkv = 65, 16
    table, nb = table_of(rng, [ctx])
    cache = R.Pool.random(rng, nb, hkv, d).to_gpu(kvq)
    (q, qt), k, v = bf(rng, 1, hkv, d), bf(rng, 1, hkv, d)[1], bf(rng, 1, hkv, d)[1]
    k[0, :, 7] = float("inf")
    acc = dev(np.ones((1, hkv, 80), np.float32))
    kvq.kvq_decode_step_accum_int8kv(cache, k, v, qt, dev(table), dev(np.array([ctx], np.int32)), ctx, 0.06, acc, split_rows=64)
    assert kvq.kvq_device_status() == 0
    pool, a = R.Pool.of(cache), acc.cpu().numpy()[0]
    page, slot = table[0, 64 // 16], 64 % 16
    assert np.isinf(pool.ks[page, :, slot]).all()
    S = np.einsum("hd,hd->h", q[0].astype(np.float64), pool.k[page, :, :, slot].reshape(hkv, d).astype(np.float64))
    pool.ks[page, :, slot] = 0.0  # its products are finite below; the key is left out there
    kf, vf, ok = pool.rows(table[0], ctx)
    ok[64] = False
    for h in range(hkv):
        if S[h] < 0:
            p, _, rel, _ = R.weights(kf[h], vf[h], ok, q[0, h:h + 1].astype(np.float64), [ctx], 0.06)
            ref = 1.0 + p[0]
            ref[64] = 0.0
            assert (np.abs(a[h, :ctx] - ref) <= rel[0] * p[0] + 2 * 2.0 ** -24 * ref).all(), h
        else:
            assert np.isnan(a[h, :ctx]).all(), h
    assert (a[:, ctx:] == 1).all()


@pytest.mark.parametrize("T,hist,keys,G,d", [
    (1, 64, [64], 2, 128), (1, 64, [64], 1, 256), (1, 300, [300], 3, 128),            # alone in its half tile
    (1, 700, list(range(640, 701)), 4, 256), (20, 1000, None, 6, 256), (130, 500, None, 2, 128),  # None: each tile's second half
    (600, 300, None, 3, 256), (1500, 0, None, 1, 128), (1200, 77, None, 2, 128)])     # keys widened once
def test_chunk_with_keys_of_nan(kvq, T, hist, keys, G, d):
    rng = np.random.default_rng(T + hist)
    hkv, n = 2, hist + T
    table, nb = table_of(rng, [n])
    pool = R.Pool.random(rng, nb, hkv, d)
    if keys is None:
        keys = np.nonzero(np.arange(n) % 128 >= 64)[0]
    set_scale(pool, table[0], keys, 1, np.nan)
    q, qt = bf(rng, T, hkv * G, d)
    acc0 = np.ones((hkv, n + 3), np.float32)
    acc = dev(acc0)
    kvq.kvq_attn_chunk_weights_int8kv(pool.to_gpu(kvq), qt, hist, dev(table[0]), 0.07, acc)
    assert kvq.kvq_device_status() == 0
    a = acc.cpu().numpy()
    assert np.isnan(a[1, :n]).all() and (a[1, n:] == 1).all()  # the last query sees every key
    one = R.Pool(*(x[:, :1] for x in (pool.k, pool.v, pool.ks, pool.vs)))
    check_chunk(one, table[0], hist, q[:, :G], acc0[:1], a[:1], 0.07)


@pytest.mark.parametrize("G,d,bad", [(1, 128, np.nan), (3, 256, np.nan), (2, 128, np.inf)])
def test_step_rows_that_are_not_finite_reach_only_the_keys_they_see(kvq, G, d, bad):
    """The first two of four query rows are not finite: the last two tokens, and the keys of a page that is not in the
    pool, are not theirs."""
    import torch
    from int8_kv_cache_quant_gb300.kvq import DEV_BAD_BLOCK
    rng = np.random.default_rng(G)
    ctx, hkv, nq = 99, 2, 4
    table, nb = table_of(rng, [ctx])
    table[0, 2] = nb + 1
    pool = R.Pool.random(rng, nb, hkv, d)
    q, qt = bf(rng, 1, nq, hkv * G, d)
    qt[0, :2, :, 5] = float(bad)
    acc = dev(np.ones((1, hkv, 112), np.float32))
    kvq.kvq_decode_step_accum_int8kv(pool.to_gpu(kvq), None, None, qt, dev(table), dev(np.array([ctx], np.int32)), ctx, 0.06, acc,
                                     split_rows=32)
    assert kvq.kvq_device_status() == DEV_BAD_BLOCK
    a = acc.cpu().numpy()[0]
    seen = np.arange(112) < ctx - 2
    seen[32:48] = False
    assert np.isnan(a[:, seen]).all() and (a[:, 32:48] == 1).all() and (a[:, ctx:] == 1).all()
    kf, vf, ok = pool.rows(table[0], ctx)
    for h in range(hkv):
        rows = q[0, 2:, h * G:(h + 1) * G].reshape(2 * G, d).astype(np.float64)
        p, _, rel, _ = R.weights(kf[h], vf[h], ok, rows, np.repeat([ctx - 1, ctx], G), 0.06)
        ref = 1.0 + p[:, ctx - 2:].sum(0)
        assert (np.abs(a[h, ctx - 2:ctx] - ref) <= (rel[:, None] * p[:, ctx - 2:]).sum(0) + (nq * G + 1) * 2.0 ** -24 * ref).all()


@pytest.mark.parametrize("T,hist", [(1000, 3000), (300, 4000)])  # keys widened once, and by each CTA
def test_rows_that_a_timeout_left_out_give_nothing_whatever_their_scores(kvq, T, hist):
    """Scores far past 2^128, whose exponential is infinite: the rows that the first run of the row pass did not finish
    (host-injected) give 0, not infinity times 0."""
    import torch
    from int8_kv_cache_quant_gb300.kvq import DEV_TIMEOUT
    rng = np.random.default_rng(T)
    hkv, G, d, scale = 1, 2, 128, 20.0
    table, nb = table_of(rng, [hist + T])
    pool = R.Pool.random(rng, nb, hkv, d)
    q, qt = bf(rng, T, G, d)
    acc = torch.zeros((1, hist + T), device="cuda")
    cache, bt = pool.to_gpu(kvq), dev(table[0])
    try:
        kvq.kvq_debug_fault_inject(4, 20_000_000)
        kvq.kvq_attn_chunk_weights_int8kv(cache, qt, hist, bt, scale, acc)
        assert kvq.kvq_device_status() == DEV_TIMEOUT
    finally:
        kvq.kvq_debug_fault_inject(0, 0)
    a = acc.double().cpu().numpy()
    # whole row tiles are gone, each other row gives 1 up to the relative error of a weight (as R.weights bounds it)
    k = pool.rows(table[0], hist + T)[0][0]
    amp = (np.abs(q.reshape(T * G, d)) @ np.abs(k).T).max() * scale * 1.4427
    rel = 4 * np.log(2) * amp * (d / 16 + 5) * 2.0 ** -23 + 4 * 2.0 ** -22 + (hist + T) * 2.0 ** -24
    assert amp > 1000 and rel < 0.1
    assert np.isfinite(a).all() and (a >= 0).all()
    kept = [T * G - x for x in range(128, T * G, 128)]
    assert min(abs(a.sum() - n) - n * rel for n in kept) <= 0, a.sum()
