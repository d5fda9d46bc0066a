"""kvq_cache_evict against an eviction by sorting: codes, scales, weights and positions to the bit."""
import numpy as np
import pytest

import forget_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def table_of(rng, lens, spare=0):
    pages = [max(1, -(-int(n) // 16)) for n in lens]
    pool = rng.permutation(sum(pages) + spare).astype(np.int32)
    table = np.full((len(lens), max(pages)), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, sum(pages) + spare


def draw_acc(rng, kind, shape):
    if kind == "spread":
        return np.exp(rng.standard_normal(shape) * 2).astype(np.float32)
    if kind == "zeros":
        return np.zeros(shape, np.float32)
    if kind == "coarse":  # many ties, -0 and +0 among them
        return (rng.integers(-2, 3, shape) * np.float32(0.5) * rng.choice([1.0, -1.0], shape)).astype(np.float32)
    a = np.exp(rng.standard_normal(shape)).astype(np.float32)  # "odd": every kind of number
    pick = rng.random(shape)
    for lo, v in ((0.0, np.nan), (0.1, np.inf), (0.15, -np.inf), (0.3, -0.0), (0.4, 0.0), (0.5, -3.5),
                  (0.55, np.finfo(np.float32).tiny / 4), (0.6, np.finfo(np.float32).max), (0.62, -np.finfo(np.float32).max)):
        a = np.where((pick >= lo) & (pick < lo + 0.05), np.float32(v), a)
    return a


def same(a, b):
    return np.array_equal(np.ascontiguousarray(a).view(np.uint32), np.ascontiguousarray(b).view(np.uint32))


def run(kvq, rng, lens, hkv, d, keep, sink, recent, kind, in_place, max_ctx=None, table=None, shuffled_pos=True, extra=0):
    import torch
    B = len(lens)
    if table is None:
        table, nb = table_of(rng, lens, spare=2)
    else:
        table, nb = table
    max_ctx = max(1, max(lens)) if max_ctx is None else max_ctx
    slots = max(table.shape[1] * 16, max_ctx)
    pool = R.Pool.random(rng, nb, hkv, d)
    acc = draw_acc(rng, kind, (B, hkv, slots + extra))
    pos = np.broadcast_to(np.arange(slots + extra, dtype=np.int32) + 100 * (sink == 0), acc.shape).copy()
    if shuffled_pos:  # a cache that has evicted before: positions in no order, the same newest for every head
        pos = rng.permuted(pos, axis=2)
    cache = pool.to_gpu(kvq)
    ga, gp, gl = dev(acc)[:, :, :slots], dev(pos)[:, :, :slots], dev(np.array(lens, np.int32))
    if in_place:
        ao, po, nl = kvq.kvq_cache_evict(cache, dev(table), gl, max_ctx, keep, ga, gp, n_sink=sink, n_recent=recent)
        assert ao is ga and po is gp
    else:
        n = min(keep, max_ctx) + 3
        ao = torch.full((B, hkv, n), -7.0, device="cuda")
        po = torch.full((B, hkv, n), -7, dtype=torch.int32, device="cuda")
        nl = torch.full((B,), -7, dtype=torch.int32, device="cuda")
        kvq.kvq_cache_evict(cache, dev(table), gl, max_ctx, keep, ga, gp, n_sink=sink, n_recent=recent, acc_out=ao,
                            slot_pos_out=po, new_lens=nl)
        assert same(ga.cpu().numpy(), acc[:, :, :slots]) and np.array_equal(gp.cpu().numpy(), pos[:, :, :slots])
    cap = min(table.shape[1] * 16, max_ctx)
    ref, outs, new = R.evict(pool, table, lens, cap, keep, sink, recent, acc, pos)
    assert np.array_equal(nl.cpu().numpy(), new)
    ao, po = ao.cpu().numpy(), po.cpu().numpy()
    for b in range(B):
        for h in range(hkv):
            ra, rp = outs[b][h]
            assert same(ao[b, h, :new[b]], ra) and np.array_equal(po[b, h, :new[b]], rp), (b, h)
            if in_place:  # nothing at or past the new length moves
                assert same(ao[b, h, new[b]:], acc[b, h, new[b]:slots]) and np.array_equal(po[b, h, new[b]:], pos[b, h, new[b]:slots])
            else:
                assert (ao[b, h, new[b]:] == -7).all() and (po[b, h, new[b]:] == -7).all()
    assert R.Pool.of(cache).same(ref)
    return kvq.kvq_device_status()


CASES = [  # lens, hkv, d, keep, sink, recent
    ([1], 1, 128, 1, 0, 0), ([2], 1, 256, 1, 0, 1), ([17], 3, 128, 16, 0, 0), ([33, 0, 16, 5], 2, 256, 16, 1, 4),
    ([100, 64, 65, 1], 2, 128, 64, 4, 60), ([257, 300], 2, 256, 250, 4, 32), ([1025] * 3, 4, 128, 1024, 4, 64),
    ([1500, 700, 31], 5, 128, 333, 0, 50), ([2049], 1, 256, 77, 2, 0), ([4100], 2, 128, 2050, 4, 100),
    ([70, 300], 300, 128, 64, 2, 8),
    ([9000], 1, 256, 1000, 4, 128), ([9000, 8193], 2, 128, 4097, 0, 999), ([12345], 1, 128, 12344, 0, 1)]


@pytest.mark.parametrize("kind", ["spread", "zeros", "coarse", "odd"])
@pytest.mark.parametrize("lens,hkv,d,keep,sink,recent", CASES)
def test_eviction(kvq, lens, hkv, d, keep, sink, recent, kind):
    rng = np.random.default_rng(len(lens) * 7919 + lens[0] + keep)
    assert run(kvq, rng, lens, hkv, d, keep, sink, recent, kind, in_place=kind in ("spread", "coarse")) == 0


def test_long_contexts_past_the_keys_in_shared_memory(kvq):
    """160 units take one CTA each: 17000 slots are more than a CTA keeps in shared memory."""
    rng = np.random.default_rng(3)
    assert run(kvq, rng, [17000] + [20] * 159, 1, 128, 9001, 4, 300, "coarse", in_place=False) == 0
    assert run(kvq, rng, [40000, 16385] + [0] * 158, 1, 128, 20, 4, 10, "spread", in_place=True) == 0
    assert run(kvq, rng, [17001] + [16400] * 2 + [3] * 157, 1, 256, 16390, 4, 300, "zeros", in_place=True) == 0


@pytest.mark.parametrize("kind,keep", [("spread", 5000), ("zeros", 70001), ("odd", 139990)])
def test_clusters_whose_ranges_pass_shared_memory(kvq, kind, keep):
    """140001 slots on eight CTAs: 17504 each."""
    rng = np.random.default_rng(6)
    assert run(kvq, rng, [140001], 1, 128, keep, 4, 300, kind, in_place=kind != "odd") == 0


def test_many_moves_in_a_large_batch(kvq):
    """160 units: up to 512 moves each without the page kernel."""
    rng = np.random.default_rng(5)
    assert run(kvq, rng, [1400, 5, 901] + [1300] * 77, 2, 128, 900, 4, 100, "spread", in_place=True) == 0
    assert run(kvq, rng, [1700, 5, 901] + [1300] * 77, 2, 128, 900, 4, 100, "spread", in_place=False) == 0


def test_rows_of_wider_arrays(kvq):
    rng = np.random.default_rng(4)
    assert run(kvq, rng, [200, 90], 2, 128, 64, 4, 8, "spread", in_place=True, extra=24) == 0
    assert run(kvq, rng, [200, 90], 1, 128, 64, 4, 8, "spread", in_place=False, extra=24) == 0


def test_lengths_past_the_bound_and_bad_pages(kvq):
    from int8_kv_cache_quant_gb300.kvq import DEV_BAD_BLOCK, DEV_BAD_POS
    rng = np.random.default_rng(9)
    # a length past max_ctx is clamped to it; a negative one counts as 0
    assert run(kvq, rng, [300, -5], 2, 128, 64, 0, 8, "spread", in_place=False, max_ctx=128) == DEV_BAD_POS
    # pages outside the pool, among the sources and among the destinations
    table, nb = table_of(rng, [320, 320])
    table[0, 1], table[0, 10], table[1, 19] = -1, nb, 1 << 30
    assert run(kvq, rng, [320, 320], 2, 256, 160, 0, 8, "spread", in_place=True, table=(table, nb)) == DEV_BAD_BLOCK
    # the same where whole pages are filled (more than 128 moves)
    table, nb = table_of(rng, [700, 699])
    table[0, 1], table[0, 30], table[1, 40] = -1, nb, 1 << 30
    assert run(kvq, rng, [700, 699], 2, 128, 300, 0, 8, "spread", in_place=True, table=(table, nb)) == DEV_BAD_BLOCK


def test_the_same_call_twice_and_on_another_stream(kvq):
    import torch
    rng = np.random.default_rng(11)
    lens, hkv, d, keep = [3000, 2500], 2, 128, 512
    table, nb = table_of(rng, lens)
    pool = R.Pool.random(rng, nb, hkv, d)
    acc = draw_acc(rng, "coarse", (2, hkv, table.shape[1] * 16))
    pos = np.broadcast_to(np.arange(acc.shape[2], dtype=np.int32), acc.shape).copy()
    args = [dev(table), dev(np.array(lens, np.int32)), max(lens), keep, dev(acc), dev(pos)]
    res = []
    for stream in (None, None, torch.cuda.Stream()):
        cache = pool.to_gpu(kvq)
        torch.cuda.synchronize()
        ao = torch.zeros((2, hkv, keep), device="cuda")
        po = torch.zeros((2, hkv, keep), dtype=torch.int32, device="cuda")
        nl = torch.zeros(2, dtype=torch.int32, device="cuda")
        ws = torch.empty(kvq.kvq_evict_workspace_bytes(2, hkv, max(lens), keep), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for _ in range(2):  # out of place, the same moves again change nothing
            kvq.kvq_cache_evict(cache, *args, n_sink=4, n_recent=64, acc_out=ao, slot_pos_out=po, new_lens=nl,
                                workspace=ws, stream=stream)
        torch.cuda.synchronize()
        res.append([t.cpu().numpy() for t in (ao, po, nl, cache.k, cache.v, cache.k_scale, cache.v_scale)])
    for r in res[1:]:
        assert all(np.array_equal(x, y) for x, y in zip(res[0], r))
    assert kvq.kvq_device_status() == 0


def test_refused_tensors(kvq):
    import torch
    c = kvq.KVCache(8, 2, 128)
    bt, ln = torch.zeros((1, 8), dtype=torch.int32, device="cuda"), torch.full((1,), 100, dtype=torch.int32, device="cuda")
    acc, pos = torch.zeros((1, 2, 128), device="cuda"), torch.zeros((1, 2, 128), dtype=torch.int32, device="cuda")
    ok = dict(cache=c, block_table=bt, ctx_lens=ln, max_ctx=100, keep=64, acc=acc, slot_pos=pos)
    for bad in (dict(acc=acc.double()), dict(acc=acc.cpu()), dict(slot_pos=pos.long()), dict(acc=acc[:, :1]),
                dict(acc=acc[:, :, :90]), dict(slot_pos=pos[:, :, :90]), dict(ctx_lens=ln.long()), dict(block_table=bt.float()),
                dict(acc_out=acc), dict(acc_out=acc[:, :, :63], slot_pos_out=pos[:, :, :63]), dict(acc=acc.expand(1, 2, 128)[:, :, ::2])):
        with pytest.raises(ValueError):
            kvq.kvq_cache_evict(**(ok | bad))
    for bad in (dict(keep=0), dict(n_sink=60, n_recent=5), dict(new_lens=ln)):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_cache_evict(**(ok | bad))
    kvq.kvq_cache_evict(**ok)
    assert kvq.kvq_device_status() == 0
