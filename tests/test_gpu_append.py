"""kvq_rope_append_int8kv to the bit: rotated q in bf16, codes and scales of k and v in their slots, and nothing
else; padding tokens, tokens out of range, pages that end inside a block, packed rows."""
import numpy as np
import pytest

import forget_ref as R
import window_ref as WR
import workloads as W
from test_gpu_evict import dev, table_of
from test_gpu_step_accum import bf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


def bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def run(kvq, rng, hq, hkv, d, seq, slot, table, nb, sections, order="chunked", ladder="shared", off=0, inter=False, far=10 ** 6,
        packed=False, stretch=1.0, flags=0, in_place=False):
    """One append against the reference; the whole cache and the rotated queries are compared to the bit."""
    import torch
    T, axes = len(seq), len(sections)
    pool = R.Pool.random(rng, nb, hkv, d)
    cache = pool.to_gpu(kvq)
    scaling = dict(scaling="yarn", factor=stretch, original_len=4096.0) if stretch > 1 else {}
    plan = kvq.kvq_rope_axes_phases(sections, base=1.0e6, order=order, ladder=ladder, **scaling)
    x = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)).to(torch.bfloat16)
    if T > 2:
        x[1, hq:] = 0  # zero rows: scale 0, codes 0
    host, x = x.float().numpy(), x.cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = rng.integers(-far, far, (axes, T)).astype(np.int32)
    layout = kvq.ROPE_INTERLEAVED if inter else kvq.ROPE_HALF
    out = q if in_place else torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = kvq.kvq_rope_append_int8kv(cache, q if hq else None, k, v, dev(pos), plan, dev(seq), dev(slot), dev(table), layout=layout,
                                     rotary_offset=off, q_out=out if hq else None)
    assert kvq.kvq_device_status() == flags
    c, s = WR.cos_sin_f32(WR.turns(pos, plan.phases.cpu().numpy().view(np.uint64), plan.axis_of), plan.attn_factor)
    kr = WR.rotate_f32(host[:, hq:hq + hkv], c, s, off, inter)
    WR.append(pool, kr, host[:, hq + hkv:], seq, slot, table)
    assert pool.same(R.Pool.of(cache))
    if hq:
        want = W.f32_to_bf16_bits(WR.rotate_f32(host[:, :hq], c, s, off, inter))
        pad = slot == -1
        assert np.array_equal(bits(got)[~pad], want[~pad])
        if not in_place:
            assert (got.float().cpu().numpy()[pad] == 7.0).all()  # a padding token's row is left as it was
    return got


SHAPES = [  # hq, hkv, d, sections, order, ladder, off, inter
    (24, 4, 256, [128], "chunked", "shared", 0, False),
    (24, 4, 256, [24, 20, 20], "turns", "shared", 64, True),
    (8, 2, 128, [24, 20, 20], "chunked", "shared", 0, False),
    (6, 6, 128, [16, 16], "chunked", "per_axis", 64, True),
    (3, 1, 256, [2, 2, 2, 2], "turns", "shared", 240, False),
    (0, 8, 128, [30, 2], "turns", "per_axis", 8, False)]


@pytest.mark.parametrize("T,first", [(1, 0), (1, 15), (5, 14), (16, 0), (16, 9), (17, 16), (31, 333), (130, 0), (700, 333)])
@pytest.mark.parametrize("hq,hkv,d,sections,order,ladder,off,inter", SHAPES)
def test_one_sequence(kvq, T, first, hq, hkv, d, sections, order, ladder, off, inter):
    rng = np.random.default_rng(T * 7 + d + hq)
    table, nb = table_of(rng, [first + T], spare=2)
    run(kvq, rng, hq, hkv, d, np.zeros(T, np.int32), np.arange(first, first + T, dtype=np.int32), table, nb, sections, order,
        ladder, off, inter, packed=T % 2 == 1, stretch=4.0 if T == 31 else 1.0)


@pytest.mark.parametrize("T,first,hq,hkv,d,sections", [(3001, 7, 24, 4, 256, [128]), (2500, 0, 7, 3, 128, [24, 20, 20]),
                                                        (9000, 16, 6, 5, 128, [8, 8]), (5000, 3, 2, 3, 256, [40, 40])])
def test_long_chunks(kvq, T, first, hq, hkv, d, sections):
    """Several KV heads a block."""
    rng = np.random.default_rng(T)
    table, nb = table_of(rng, [first + T], spare=2)
    run(kvq, rng, hq, hkv, d, np.zeros(T, np.int32), np.arange(first, first + T, dtype=np.int32), table, nb, sections, packed=True)


@pytest.mark.parametrize("d", [128, 256])
def test_a_ragged_batch_with_padding(kvq, d):
    """Several sequences' new tokens behind each other, padding between and behind them, slots in any order."""
    rng = np.random.default_rng(d)
    lens = [1, 40, 200, 17, 64]
    table, nb = table_of(rng, [n + 30 for n in lens], spare=3)
    seq, slot = [], []
    for b, n in enumerate(lens):
        at = int(rng.integers(0, 30))
        seq += [b] * n + [0] * 3
        slot += list(range(at, at + n)) + [-1] * 3
    seq, slot = np.array(seq, np.int32), np.array(slot, np.int32)
    seq[slot == -1] = 99  # not looked at
    run(kvq, rng, 8, 2, d, seq, slot, table, nb, [40, 12, 12], "chunked")
    order = rng.permutation(len(seq))
    run(kvq, rng, 8, 2, d, seq[order], slot[order], table, nb, [40, 12, 12], "turns", packed=True, in_place=True)
    run(kvq, rng, 8, 2, d, seq, np.full(len(seq), -1, np.int32), table, nb, [40, 12, 12])


def test_tokens_out_of_range(kvq):
    rng = np.random.default_rng(9)
    table, nb = table_of(rng, [50, 50])
    table[1, 2] = nb + 4
    cases = [([0, 2, 1], [3, 4, 5], kvq.kvq.DEV_BAD_SEQ), ([0, -1, 1], [3, 4, 5], kvq.kvq.DEV_BAD_SEQ),
             ([0, 0, 1], [3, 16 * table.shape[1], 5], kvq.kvq.DEV_BAD_POS), ([0, 0, 1], [3, -2, 5], kvq.kvq.DEV_BAD_POS),
             ([0, 0, 1], [2 ** 31 - 1, 6, 5], kvq.kvq.DEV_BAD_POS), ([0, 0, 1], [3, 4, 33], kvq.kvq.DEV_BAD_BLOCK)]
    for seq, slot, flag in cases:
        run(kvq, rng, 4, 2, 128, np.array(seq, np.int32), np.array(slot, np.int32), table, nb, [64], flags=flag)


def test_rows_that_are_not_finite(kvq):
    """As kvq_quant_write stores them: the rotation that leaves rows as they are, then the same codes and scales."""
    import torch
    rng = np.random.default_rng(10)
    x, t = bf(rng, 6, 2, 128)
    for i, bad in enumerate((np.inf, -np.inf, np.nan)):
        t[i, 0, 5 * i + 3] = bad
    t[3, 0] = float("nan")
    t[4, 1, :64], t[4, 1, 64:] = float("nan"), 0.0
    table, nb = table_of(rng, [6])
    a, b = kvq.KVCache(nb, 2, 128), kvq.KVCache(nb, 2, 128)
    seq, slot = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.arange(6, dtype=torch.int32, device="cuda")
    kvq.kvq_quant_write(a, t, t, seq, slot, dev(table))
    plan = kvq.kvq_rope_axes_phases([8])
    kvq.kvq_rope_append_int8kv(b, None, t, t, torch.zeros_like(slot), plan, seq, slot, dev(table))
    # an angle of 0 takes x to x 1 - y 0: NaN where the partner is not finite, so k is compared outside the rotated part's rows
    assert torch.equal(a.v, b.v) and torch.equal(a.v_scale.view(torch.int32), b.v_scale.view(torch.int32))
    assert torch.equal(a.k[..., 5, :], b.k[..., 5, :])


def test_far_page_of_a_large_pool(kvq):
    """Pages whose codes lie past 2 GB and past 4 GB."""
    import torch
    rng = np.random.default_rng(11)
    hkv, d, nb = 8, 256, 140000  # 4.6 GB of codes a side
    cache = kvq.KVCache(nb, hkv, d)
    table = np.array([[70000, nb - 1]], np.int32)
    x, t = bf(rng, 20, hkv, d)
    seq, slot = torch.zeros(20, dtype=torch.int32, device="cuda"), torch.arange(8, 28, dtype=torch.int32, device="cuda")
    plan = kvq.kvq_rope_axes_phases([32])
    kvq.kvq_rope_append_int8kv(cache, None, t, t, torch.zeros_like(slot), plan, seq, slot, dev(table))
    code, scale = WR.quantise(x)
    for i in range(20):
        page, at = table[0, (8 + i) // 16], (8 + i) % 16
        assert np.array_equal(cache.v[page, :, :, at].cpu().numpy(), code[i])
        assert np.array_equal(cache.k[page, :, :, at].cpu().numpy().reshape(hkv, d), code[i])
        assert np.array_equal(cache.v_scale[page, :, at].cpu().numpy(), scale[i])


def test_capture_replays(kvq):
    import torch
    rng = np.random.default_rng(12)
    table, nb = table_of(rng, [64])
    q, k, v = (bf(rng, 3, h, 128)[1] for h in (8, 2, 2))
    plan = kvq.kvq_rope_axes_phases([24, 20, 20])
    pos, seq = torch.zeros((3, 3), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    slot, bt = torch.arange(3, dtype=torch.int32, device="cuda"), dev(table)
    a, b = kvq.KVCache(nb, 2, 128), kvq.KVCache(nb, 2, 128)
    out = kvq.kvq_rope_append_int8kv(a, q, k, v, pos, plan, seq, slot, bt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_rope_append_int8kv(a, q, k, v, pos, plan, seq, slot, bt, q_out=out)
    kvq.kvq_rope_append_int8kv(b, q, k, v, pos, plan, seq, slot, bt)
    slot += 14
    pos += 5
    graph.replay()
    want = kvq.kvq_rope_append_int8kv(b, q, k, v, pos, plan, seq, slot, bt)
    assert torch.equal(out, want)
    assert all(torch.equal(x, y) for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)))
    assert kvq.kvq_device_status() == 0
