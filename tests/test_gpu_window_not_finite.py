"""Rows that hold infinities and NaN, in the calls around windowed attention: what becomes of the rows themselves."""
import numpy as np
import pytest

import forget_ref as R
import window_ref as WR
from test_gpu_evict import dev, table_of
from test_gpu_step_accum import bf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("force", [1, 2])
@pytest.mark.parametrize("hq,hkv,d,new", [(8, 2, 128, 3), (24, 4, 256, 1), (24, 4, 256, 4), (8, 2, 128, 1)])
def test_a_query_row_of_the_step(kvq, bad, force, hq, hkv, d, new):
    """NaN in its own outputs (an infinite element gives scores of both infinities), all of them, and in no others."""
    import torch
    rng = np.random.default_rng(7)
    table, nb = table_of(rng, [500])
    pool = R.Pool.random(rng, nb, hkv, d)
    q = bf(rng, 1, new, hq, d)[1]
    call = lambda: kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), None, None, q, dev(table), dev(np.array([500], np.int32)), 500,  # noqa: E731
                                                     0.1, 100, 4, force_route=force)
    want = call()
    q[0, new // 2, 3, 7] = bad
    got = call()
    mine = torch.zeros((new, hq), dtype=torch.bool, device="cuda")
    mine[new // 2, 3] = True
    assert torch.equal(got[0][~mine], want[0][~mine]) and torch.isnan(got[0][mine]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("hq,hkv,d,T,history", [(8, 2, 256, 100, 600), (32, 8, 128, 400, 300), (8, 1, 128, 1, 1000)])
def test_a_query_row_of_a_chunk(kvq, bad, hq, hkv, d, T, history):
    import torch
    rng = np.random.default_rng(8)
    table, nb = table_of(rng, [history + T])
    pool = R.Pool.random(rng, nb, hkv, d)
    q = bf(rng, T, hq, d)[1]
    for dtype in (torch.bfloat16, torch.float32):
        x = q.clone()
        call = lambda: kvq.kvq_attn_prefill_window_int8kv(pool.to_gpu(kvq), x, history, dev(table[0]), 0.06, 150, 4, out_dtype=dtype)  # noqa: E731
        want = call()
        x[T // 2, 0, 9] = bad
        got = call()
        mine = torch.zeros((T, hq), dtype=torch.bool, device="cuda")
        mine[T // 2, 0] = True
        assert torch.equal(got[~mine], want[~mine]) and torch.isnan(got[mine].float()).all()


def codes_of(x):
    """The rule of kvq_quant_write on fp32 rows, non-finite ones too: the largest magnitude is of the numbers among them, and a
    quotient that is no number has code -127."""
    amax = np.fmax.reduce(np.abs(x), -1, initial=np.float32(0.0)).astype(np.float32)
    scale = (amax / np.float32(127.0)).astype(np.float32)
    with np.errstate(all="ignore"):
        q = (x / scale[..., None]).astype(np.float32)
    code = np.where(np.isnan(q), -127.0, np.clip(np.rint(np.where(np.isnan(q), 0.0, q)), -127, 127))
    return np.where(amax[..., None] > 0, code, 0.0).astype(np.int8), scale


@pytest.mark.parametrize("d,inter,off", [(128, False, 0), (256, True, 64), (128, True, 0), (256, False, 128)])
def test_rows_of_the_append(kvq, d, inter, off):
    """K and V codes and scales of rows that are not finite, in the rotated dims and outside of them, against the rule, and V and
    the K rows that the rotation leaves as they are against kvq_quant_write."""
    import torch
    rng = np.random.default_rng(10)
    T, hkv, r = 24, 2, 32
    x, t = bf(rng, T, hkv, d)
    t = t.clone()
    out_of = [i for i in range(d) if not off <= i < off + r]  # dims that the rotation leaves
    for i, bad in enumerate((np.inf, -np.inf, np.nan) * 2):
        t[i, 0, off + 5 * i + 3] = bad               # a rotated dim
        t[6 + i, 1, out_of[11 * i + 2]] = bad        # another
        t[12 + i, 0, out_of[7 * i]], t[12 + i, 0, out_of[7 * i + 1]] = bad, -bad
    t[18, 0] = float("nan")
    t[19, 1, :64], t[19, 1, 64:] = float("nan"), 0.0
    t[20, 0], t[20, 0, out_of[3]] = 0.0, float("nan")
    t[21, 1, off:off + r], t[21, 1, off + 2] = 0.0, float("inf")
    t[22, 0], t[23, 1] = float("inf"), float("-inf")
    x = t.float().cpu().numpy()
    table, nb = table_of(rng, [T])
    a, b = kvq.KVCache(nb, hkv, d), kvq.KVCache(nb, hkv, d)
    seq, slot = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    kvq.kvq_quant_write(a, t, t, seq, slot, dev(table))
    plan = kvq.kvq_rope_axes_phases([r // 2])
    pos = rng.integers(1, 10 ** 6, T).astype(np.int32)
    kvq.kvq_rope_append_int8kv(b, None, t, t, dev(pos), plan, seq, slot, dev(table), rotary_offset=off,
                               layout=kvq.ROPE_INTERLEAVED if inter else kvq.ROPE_HALF)
    assert torch.equal(a.v, b.v) and torch.equal(a.v_scale.view(torch.int32), b.v_scale.view(torch.int32))
    c, s = WR.cos_sin_f32(WR.turns(pos[None], plan.phases.cpu().numpy().view(np.uint64), plan.axis_of), plan.attn_factor)
    with np.errstate(all="ignore"):
        code, scale = codes_of(WR.rotate_f32(x, c, s, off, inter))
    got = R.Pool.of(b)
    page, at = table[0, np.arange(T) // 16], np.arange(T) % 16
    assert np.array_equal(got.k[page, :, :, at].reshape(T, hkv, d), code)
    assert np.array_equal(got.ks[page, :, at].view(np.int32), scale.view(np.int32))
    # a position of 0 leaves finite pairs as they are: the rows whose rotated dims are finite are those of kvq_quant_write
    kvq.kvq_rope_append_int8kv(b, None, t, t, torch.zeros_like(slot), plan, seq, slot, dev(table), rotary_offset=off,
                               layout=kvq.ROPE_INTERLEAVED if inter else kvq.ROPE_HALF)
    plain, got = R.Pool.of(a), R.Pool.of(b)
    i, h = np.nonzero(np.isfinite(x[..., off:off + r]).all(-1))
    assert len(i) > T and np.array_equal(got.k[page[i], h, :, at[i]], plain.k[page[i], h, :, at[i]])
    assert np.array_equal(got.ks[page[i], h, at[i]].view(np.int32), plain.ks[page[i], h, at[i]].view(np.int32))
    assert kvq.kvq_device_status() == 0
