"""kvq_attn_prefill_window_int8kv over the whole range of V scales that it takes, against fp64: rows of zeros (scale 0) beside
rows of large values, whichever comes first; scales past the range are reported."""
import numpy as np
import pytest

import forget_ref as R
import window_ref as WR
from test_gpu_evict import dev, table_of
from test_gpu_prefill_window import run
from test_gpu_step_accum import bf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


def keys_of(table, n):
    """(pages, slots) of keys 0 .. n - 1."""
    t = np.arange(n)
    return table[0, t // 16], t % 16


WHERE = {"between": lambda n: np.arange(n) % 3 == 1, "first": lambda n: np.arange(n) < n // 2, "last": lambda n: np.arange(n) >= n // 2}


@pytest.mark.parametrize("where", list(WHERE))
@pytest.mark.parametrize("bits", [20, 27, 39])
@pytest.mark.parametrize("T,history,hq,hkv,d", [(40, 300, 8, 2, 128), (300, 500, 6, 1, 256)])
def test_zero_rows_beside_large_ones(kvq, where, bits, T, history, hq, hkv, d):
    """A row of zeros takes its part of the softmax's sum however large the other V rows are."""
    rng = np.random.default_rng(bits)
    n = history + T

    def edit(pool, table):
        zero = WHERE[where](n)
        page, at = keys_of(table, n)
        pool.vs[page, :, at] = np.where(zero, 0.0, 2.0 ** (bits + rng.uniform(0, 1, n)))[:, None]
        pool.v[page[zero], :, :, at[zero]] = 0

    run(kvq, rng, T, history, hq, hkv, d, 5000, 0, edit=edit)
    run(kvq, rng, T, history, hq, hkv, d, 150, 20, edit=edit, scale=1e-6)  # all scores alike


@pytest.mark.parametrize("d", [128, 256])
def test_the_range_of_scales(kvq, d):
    """Scales from 2^-60 to 2^40, all scores alike and not."""
    rng = np.random.default_rng(d)

    def edit(pool, table):
        pool.vs[:] = 2.0 ** rng.uniform(-60, 40, pool.vs.shape)

    for scale in (1e-6, None, 0.5):
        run(kvq, rng, 150, 500, 8, 2, d, 400, 20, edit=edit, scale=scale)


def test_two_keys(kvq):
    """Two keys with equal scores, V of one zero: half of the other's V."""
    import torch
    for bits in (0, 26, 27, 39):
        pool = R.Pool.random(np.random.default_rng(1), 1, 1, 128)
        pool.ks[:] = 0.0
        pool.vs[0, 0, :2] = 0.0, 2.0 ** bits
        pool.v[0, :, :, 0], pool.v[0, :, :, 1] = 0, 64
        out = kvq.kvq_attn_prefill_window_int8kv(pool.to_gpu(kvq), bf(np.random.default_rng(2), 1, 1, 128)[1], 1, dev(np.zeros(1, np.int32)),
                                                 0.1, 16, out_dtype=torch.float32)
        # the logarithms of both scales are within a step of fp32, 2^-18 below 64, which is ln 2 of it in a weight each; the rest
        # is some steps of 2^-22
        assert np.abs(out.cpu().numpy() / 2.0 ** bits - 32.0).max() <= 32 * (2 * np.log(2) * 2.0 ** -18 + 2.0 ** -20)
    assert kvq.kvq_device_status() == 0


@pytest.mark.parametrize("large", [2.0 ** 41, 3.0e38, float("inf")])
def test_a_scale_past_the_range_is_reported(kvq, large):
    """On a key that some query sees; a hidden one may hold anything."""
    rng = np.random.default_rng(3)
    table, nb = table_of(rng, [300])
    q, row = bf(rng, 10, 8, 128)[1], dev(table[0])
    for key, flags in ((280, kvq.kvq.DEV_BAD_SCALE), (3, kvq.kvq.DEV_BAD_SCALE), (241, kvq.kvq.DEV_BAD_SCALE), (240, 0), (4, 0)):
        pool = R.Pool.random(rng, nb, 2, 128)
        pool.vs[table[0, key // 16], 1, key % 16] = large
        kvq.kvq_attn_prefill_window_int8kv(pool.to_gpu(kvq), q, 290, row, 0.1, 50, 4)
        assert kvq.kvq_device_status() == flags, key


@pytest.mark.parametrize("octaves", [0.6, 12.3, 18.7, 22.4, 25.6, 29.5])
def test_small_weights(kvq, octaves):
    """One key far above the others, all of whose weights are the same, in dims where it has a code of 0: a weight goes in as fp16, off
    by 2^-11 of itself or 2^-32 of the row's largest."""
    import torch
    rng = np.random.default_rng(4)
    d, n, scale = 128, 1000, 0.125
    table, nb = table_of(rng, [n])
    pool = R.Pool.random(rng, nb, 1, d)
    pool.vs[:], pool.ks[:], pool.k[:] = 1.0, 1.0, 0
    page, at = keys_of(table, n)
    top = 200
    pool.k[page[top], 0, 0, at[top], 0], pool.ks[page[top], 0, at[top]] = 64, octaves * np.log(2) / (64 * scale)
    pool.v[page[top], 0, ::2, at[top]] = 0
    q = torch.ones((1, 4, d), dtype=torch.bfloat16, device="cuda")
    out = kvq.kvq_attn_prefill_window_int8kv(pool.to_gpu(kvq), q, n - 1, dev(table[0]), scale, 5000, out_dtype=torch.float32)
    ref, _ = WR.prompt(pool, table[0], np.ones((1, 4, d)), n - 1, 5000, 0, scale)
    v = np.abs(pool.rows(table[0], n)[1][0])
    p = np.where(np.arange(n) == top, 1.0, 2.0 ** -octaves)
    p /= p.sum()
    # the score: two factors' roundings and the sum's, 2^-22 of it in octaves; weights, sum and quotient some steps more
    rel = np.log(2) * octaves * 2.0 ** -22 + 2.0 ** -20 + n * 2.0 ** -24
    tol = (p @ v) * rel + np.maximum(2.0 ** -11 * p, 2.0 ** -32 * p.max()) @ v
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()
