"""kvq_decode_step_accum_int8kv: the output of the decode step, and every key's accumulated weight
against fp64; the cache writes and positions to the bit; failures; and the loop of rotation, step and
eviction as a serving program runs it."""
import numpy as np
import pytest

import forget_ref as R
from test_gpu_evict import dev, same, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


def bf(rng, *shape):
    """bf16 values as fp32 numpy, and the tensor."""
    import torch
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()
    return t.float().cpu().numpy(), t


def check(pool, table, lens, cap, q, out, acc0, acc, hkv, scale, wrote, n_new):
    """Output and weights of every sequence, from the codes that are in the cache after the call."""
    B, nq, Hq, D = q.shape
    G = Hq // hkv
    for b in range(B):
        n = max(0, min(int(lens[b]), cap))
        k, v, ok = pool.rows(table[b], n)
        for h in range(hkv):
            rows = q[b, :, h * G:(h + 1) * G].reshape(nq * G, D).astype(np.float64)
            lim = np.repeat(n - nq + 1 + np.arange(nq), G)
            p, o, rel, mag = R.weights(k[h], v[h], ok, rows, lim, scale)
            got = out[b, :, h * G:(h + 1) * G].reshape(nq * G, D)
            # the softmax weight goes in as two fp16 parts (2^-22), O is summed over n keys and the splits
            assert (np.abs(got - o) <= (rel[:, None] + 2.0 ** -22 + n * 2.0 ** -24) * mag + 1e-30).all(), (b, h)
            fresh = acc0[b, h, :n].astype(np.float64)
            if wrote[b]:
                fresh[n - n_new:] = 0.0
            ref = fresh + p.sum(0)
            # the rows' sum and the addition to what was there round R + 1 times
            tol = (rel[:, None] * p).sum(0) + (len(lim) + 1) * 2.0 ** -24 * np.abs(ref) + 1e-30
            assert (np.abs(acc[b, h, :n] - ref) <= tol).all(), (b, h, np.abs(acc[b, h, :n] - ref).max())
            assert same(acc[b, h, n:], acc0[b, h, n:])  # entries past the sequence


CASES = [  # lens, hkv, G, d, n_new, split
    ([1], 1, 1, 128, 1, 0), ([1], 2, 6, 256, 1, 0), ([16, 17, 15], 2, 4, 128, 1, 0), ([40, 0, 200], 1, 8, 256, 1, 16),
    ([700, 333], 4, 6, 256, 1, 0), ([1024], 4, 6, 256, 1, 64), ([1500, 64, 1], 2, 3, 128, 1, 0), ([555], 1, 16, 128, 1, 0),
    ([300, 5], 2, 6, 256, 4, 0), ([129, 700], 1, 8, 128, 5, 48), ([90], 1, 1, 256, 7, 16), ([260], 2, 16, 128, 3, 0),
    ([2000, 1999], 1, 12, 256, 2, 0)]


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("lens,hkv,G,d,n_new,split", CASES)
def test_step(kvq, lens, hkv, G, d, n_new, split, write):
    run_step(kvq, lens, hkv, G, d, n_new, split, write)


@pytest.mark.parametrize("lens,hkv,G,d,n_new,split,extra", [
    ([300] * 22 + [1, 17], 4, 6, 256, 1, 0, 0), ([90] * 40 + [33], 2, 8, 128, 1, 16, 0),  # a merging warp a row
    ([165000], 1, 1, 128, 1, 16, 0),                                            # 10313 splits
    ([1030, 555], 3, 2, 128, 2, 0, 1), ([1030, 555], 3, 2, 256, 1, 0, 2), ([4097], 2, 1, 128, 1, 0, 3)])  # odd rows of acc
def test_step_in_its_other_launches(kvq, lens, hkv, G, d, n_new, split, extra):
    run_step(kvq, lens, hkv, G, d, n_new, split, True, extra)


def run_step(kvq, lens, hkv, G, d, n_new, split, write, extra=0):
    import torch
    rng = np.random.default_rng(lens[0] * 31 + hkv * 7 + G + d + n_new)
    B = len(lens)
    table, nb = table_of(rng, lens)
    pool = R.Pool.random(rng, nb, hkv, d)
    cache = pool.to_gpu(kvq)
    max_ctx, slots = max(lens), table.shape[1] * 16 + extra
    q, qt = bf(rng, B, n_new, hkv * G, d)
    kn, vn = bf(rng, B, n_new, hkv, d)[1], bf(rng, B, n_new, hkv, d)[1]
    acc0 = np.exp(rng.standard_normal((B, hkv, slots))).astype(np.float32)
    pos0 = rng.integers(0, 1 << 30, (B, hkv, slots)).astype(np.int32)
    first = rng.integers(0, 1 << 20, B).astype(np.int32)
    acc, sp, pos, ctx = dev(acc0), dev(pos0), dev(first), dev(np.array(lens, np.int32))
    scale = 1.0 / np.sqrt(d)
    wrote = [write and n >= n_new for n in lens]
    # what the step without weights does to the same cache and queries
    twin = pool.to_gpu(kvq)
    if write:
        ref = kvq.kvq_decode_step_int8kv(twin, kn, vn, qt, dev(table), ctx, max_ctx, scale, split_rows=split, force_route=2)
        flags = kvq.kvq_device_status()
        out = kvq.kvq_decode_step_accum_int8kv(cache, kn, vn, qt, dev(table), ctx, max_ctx, scale, acc, slot_pos=sp, pos=pos,
                                               split_rows=split)
    else:
        ref = kvq.kvq_attn_verify_int8kv(twin, qt, dev(table), ctx, max_ctx, scale, split_rows=split, force_route=2)
        flags = kvq.kvq_device_status()
        out = kvq.kvq_decode_step_accum_int8kv(cache, None, None, qt, dev(table), ctx, max_ctx, scale, acc, split_rows=split)
    assert kvq.kvq_device_status() == flags == (0 if not write or all(wrote) else kvq.kvq.DEV_BAD_POS)
    assert torch.equal(out, ref)
    assert R.Pool.of(cache).same(R.Pool.of(twin))
    spn = sp.cpu().numpy()
    for b, n in enumerate(lens):
        want = pos0[b].copy()
        if wrote[b]:
            want[:, n - n_new:n] = first[b] + np.arange(n_new)
        assert np.array_equal(spn[b], want)
    check(R.Pool.of(cache), table, lens, max_ctx, q, out.cpu().numpy(), acc0, acc.cpu().numpy(), hkv, scale, wrote, n_new)


def test_weights_of_a_row_sum_to_one(kvq):
    """Over a long context with the automatic split: each row gives weight 1 in all."""
    import torch
    rng = np.random.default_rng(2)
    lens, hkv, G, d = [20000, 4097], 2, 4, 128
    table, nb = table_of(rng, lens)
    cache = R.Pool.random(rng, nb, hkv, d).to_gpu(kvq)
    acc = torch.zeros((2, hkv, table.shape[1] * 16), device="cuda")
    qt = bf(rng, 2, hkv * G, d)[1]
    kvq.kvq_decode_step_accum_int8kv(cache, None, None, qt, dev(table), dev(np.array(lens, np.int32)), max(lens), 0.05, acc)
    s = acc.double().sum(2).cpu().numpy()
    # l and each weight carry the fp32 errors that R.weights bounds; n 2^-24 for l is the largest
    assert np.abs(s - G).max() <= G * (20000 * 2.0 ** -24 + 1e-5)
    assert (acc[1, :, 4097:] == 0).all()


def test_lengths_past_the_bound_and_bad_pages(kvq):
    import torch
    from int8_kv_cache_quant_gb300.kvq import DEV_BAD_BLOCK, DEV_BAD_POS
    rng = np.random.default_rng(21)
    lens, hkv, G, d = [96, 300, 64], 2, 4, 256
    table, nb = table_of(rng, lens)
    table[0, 2], table[2, 0] = nb + 5, -9
    pool = R.Pool.random(rng, nb, hkv, d)
    acc0 = np.ones((3, hkv, table.shape[1] * 16), np.float32)
    q, qt = bf(rng, 3, 1, hkv * G, d)
    kn, vn = bf(rng, 3, 1, hkv, d)[1], bf(rng, 3, 1, hkv, d)[1]
    cache, acc = pool.to_gpu(kvq), dev(acc0)
    sp, pos = torch.zeros(acc.shape, dtype=torch.int32, device="cuda"), torch.full((3,), 7, dtype=torch.int32, device="cuda")
    out = kvq.kvq_decode_step_accum_int8kv(cache, kn, vn, qt, dev(table), dev(np.array(lens, np.int32)), 128, 0.06, acc,
                                           slot_pos=sp, pos=pos)
    # sequence 1 is longer than max_ctx: attended up to it, nothing written, no entry set
    assert kvq.kvq_device_status() == DEV_BAD_BLOCK | DEV_BAD_POS
    check(R.Pool.of(cache), table, lens, 128, q, out.cpu().numpy(), acc0, acc.cpu().numpy(), hkv, 0.06, [True, False, True], 1)
    assert (sp[1] == 0).all() and (sp[0, :, 95] == 7).all()
    bad = acc.cpu().numpy()
    assert (bad[0, :, 32:48] == 1).all() and (bad[2, :, :16] == 1).all()  # keys of the bad pages gain nothing


def test_a_range_that_ran_out_of_time_gives_no_weight(kvq):
    """The bounded wait of the first range runs out (host-injected): the call returns, the status says so,
    the range's keys gain nothing and the others' weights still sum to 1 per row."""
    import torch
    from int8_kv_cache_quant_gb300.kvq import DEV_TIMEOUT
    rng = np.random.default_rng(22)
    lens, hkv, G, d = [1024], 1, 4, 256
    table, nb = table_of(rng, lens)
    cache = R.Pool.random(rng, nb, hkv, d).to_gpu(kvq)
    acc = torch.zeros((1, hkv, 1024), device="cuda")
    qt = bf(rng, 1, G, d)[1]
    args = (cache, None, None, qt, dev(table), dev(np.array(lens, np.int32)), 1024, 0.06, acc)
    try:
        kvq.kvq_debug_fault_inject(1, 20_000_000)
        kvq.kvq_decode_step_accum_int8kv(*args, split_rows=256)
        assert kvq.kvq_device_status() == DEV_TIMEOUT
    finally:
        kvq.kvq_debug_fault_inject(0, 0)
    a = acc.cpu().numpy().astype(np.float64)
    assert (a[0, 0, :256] == 0).all() and abs(a.sum() - G) < 1e-4
    acc.zero_()
    kvq.kvq_decode_step_accum_int8kv(*args, split_rows=256)
    assert kvq.kvq_device_status() == 0 and abs(float(acc.double().sum()) - G) < 1e-4


def test_refused_tensors(kvq):
    import torch
    c = kvq.KVCache(8, 2, 128)
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    kn = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    bt, ln = torch.zeros((1, 8), dtype=torch.int32, device="cuda"), torch.full((1,), 100, dtype=torch.int32, device="cuda")
    acc, sp = torch.zeros((1, 2, 128), device="cuda"), torch.zeros((1, 2, 128), dtype=torch.int32, device="cuda")
    ok = dict(cache=c, k_new=kn, v_new=kn, q=q, block_table=bt, ctx_lens=ln, max_ctx=100, softmax_scale=0.1, acc=acc,
              slot_pos=sp, pos=ln)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(acc=acc[:, :1]), dict(acc=acc[:, :, :99]), dict(acc=acc.half()),
                dict(slot_pos=sp.long()), dict(pos=None), dict(k_new=kn.float()), dict(k_new=torch.cat([kn, kn])),
                dict(ctx_lens=ln.long()), dict(ctx_lens=ln.expand(2)), dict(block_table=bt[:, ::2])):
        with pytest.raises(ValueError):
            kvq.kvq_decode_step_accum_int8kv(**(ok | bad))
    for bad in (dict(v_new=None), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_decode_step_accum_int8kv(**(ok | bad))


def test_graph_replay(kvq):
    """A step and an eviction captured once and replayed: the bits of the eager calls, on new inputs too."""
    import torch
    rng = np.random.default_rng(31)
    lens, hkv, G, d, keep = [513, 513], 2, 4, 128, 512
    table, nb = table_of(rng, lens)
    pool = R.Pool.random(rng, nb, hkv, d)
    slots = table.shape[1] * 16
    acc0 = np.exp(rng.standard_normal((2, hkv, slots))).astype(np.float32)
    pos0 = np.broadcast_to(np.arange(slots, dtype=np.int32), acc0.shape).copy()

    class Side:
        def __init__(self):
            self.cache, self.acc, self.sp = pool.to_gpu(kvq), dev(acc0), dev(pos0)
            self.q, self.k, self.v = (torch.empty((2, h, d), dtype=torch.bfloat16, device="cuda") for h in (hkv * G, hkv, hkv))
            self.table, self.ctx, self.pos = dev(table), dev(np.array(lens, np.int32)), dev(np.array([513, 513], np.int32))
            self.out, self.nl = torch.empty((2, hkv * G, d), device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
            self.w1 = torch.empty(kvq.kvq_step_accum_workspace_bytes(2, 1, hkv * G, 513, d), dtype=torch.uint8, device="cuda")
            self.w2 = torch.empty(kvq.kvq_evict_workspace_bytes(2, hkv, 513, keep), dtype=torch.uint8, device="cuda")

        def load(self, seed):
            g = torch.Generator(device="cuda").manual_seed(seed)
            for t in (self.q, self.k, self.v):
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

        def call(self):
            kvq.kvq_decode_step_accum_int8kv(self.cache, self.k, self.v, self.q, self.table, self.ctx, 513, 0.1, self.acc,
                                             slot_pos=self.sp, pos=self.pos, out=self.out, workspace=self.w1)
            kvq.kvq_cache_evict(self.cache, self.table, self.ctx, 513, keep, self.acc, self.sp, n_sink=2, n_recent=16,
                                new_lens=self.nl, workspace=self.w2)
            self.pos += 1

        def state(self):
            return [t.cpu().numpy() for t in (self.out, self.acc, self.sp, self.nl, self.cache.k, self.cache.v,
                                              self.cache.k_scale, self.cache.v_scale)]

    eager, graphed = Side(), Side()
    for s in (eager, graphed):
        s.load(0)
        s.call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.call()
    for seed in (1, 2, 3):
        for s in (eager, graphed):
            s.load(seed)
        eager.call()
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a, b) for a, b in zip(eager.state(), graphed.state())), seed
    assert kvq.kvq_device_status() == 0


def test_the_serving_loop(kvq):
    """Rotation by position, step, eviction, over and over within one budget: every call is checked from
    the state it found, and at the end the newest tokens are still there and the sinks too."""
    import torch
    rng = np.random.default_rng(41)
    B, hkv, G, d, keep, sink, recent = 2, 2, 3, 128, 48, 2, 8
    room = keep + 16
    table, nb = table_of(rng, [room] * B)
    pool = R.Pool.random(rng, nb, hkv, d)
    cache = pool.to_gpu(kvq)
    acc, sp = torch.zeros((B, hkv, room), device="cuda"), torch.zeros((B, hkv, room), dtype=torch.int32, device="cuda")
    bt, ph = dev(table), kvq.kvq_rope_phases(64, 1.0e4)[0]
    lens = np.zeros(B, np.int32)
    scale = 1.0 / np.sqrt(d)
    for step in range(150):
        lens = lens + 1
        pos = dev(np.full(B, step, np.int32))
        q, k = kvq.kvq_rope_bf16(bf(rng, B, hkv * G, d)[1], bf(rng, B, hkv, d)[1], pos, ph)
        v = bf(rng, B, hkv, d)[1]
        a0 = acc.cpu().numpy()
        ctx = dev(lens)
        out = kvq.kvq_decode_step_accum_int8kv(cache, k, v, q, bt, ctx, room, scale, acc, slot_pos=sp, pos=pos)
        a1 = acc.cpu().numpy()
        check(R.Pool.of(cache), table, lens, room, q.float().cpu().numpy()[:, None], out.cpu().numpy()[:, None], a0, a1, hkv,
              scale, [True] * B, 1)
        if lens[0] == room or step % 13 == 12:
            before, p1 = R.Pool.of(cache), sp.cpu().numpy()
            _, _, nl = kvq.kvq_cache_evict(cache, bt, ctx, room, keep, acc, sp, n_sink=sink, n_recent=recent)
            ref, outs, lens = R.evict(before, table, lens, room, keep, sink, recent, a1, p1)
            assert np.array_equal(nl.cpu().numpy(), lens) and R.Pool.of(cache).same(ref)
            a2, p2 = acc.cpu().numpy(), sp.cpu().numpy()
            for b in range(B):
                for h in range(hkv):
                    assert same(a2[b, h, :lens[b]], outs[b][h][0]) and np.array_equal(p2[b, h, :lens[b]], outs[b][h][1])
            held = p2[:, :, :lens[0]]
            for b in range(B):
                for h in range(hkv):
                    have = set(held[b, h].tolist())
                    assert len(have) == lens[b] and {0, 1} <= have
                    assert set(range(max(0, step - recent + 1), step + 1)) <= have
    assert kvq.kvq_device_status() == 0


def test_pages_past_two_gigabytes(kvq):
    """The same calls on pages at the end of a pool whose K passes 2^31 bytes: the bits of a small pool."""
    import torch
    rng = np.random.default_rng(43)
    hkv, G, d, T, hist, keep = 4, 6, 256, 300, 900, 500
    n = hist + T
    table, nb = table_of(rng, [n + 1])
    small = R.Pool.random(rng, nb, hkv, d).to_gpu(kvq)
    far = (1 << 31) // (hkv * d * 16) + 100 - nb
    big = kvq.KVCache.wrap(*(torch.empty((far + nb,) + t.shape[1:], dtype=t.dtype, device="cuda")
                             for t in (small.k, small.v, small.k_scale, small.v_scale)))
    for t, u in zip((big.k, big.v, big.k_scale, big.v_scale), (small.k, small.v, small.k_scale, small.v_scale)):
        t[far:] = u
    q, k, v = (bf(rng, T, h, d)[1] for h in (hkv * G, hkv, hkv))
    slots = table.shape[1] * 16
    res = []
    for cache, first in ((small, 0), (big, far)):
        bt = dev((table + first).astype(np.int32))
        acc = torch.zeros((1, hkv, slots), device="cuda")
        sp = torch.arange(slots, dtype=torch.int32, device="cuda").repeat(1, hkv, 1)
        for rows in (1, 20, T):  # one row tile, a few, and keys widened once
            kvq.kvq_attn_chunk_weights_int8kv(cache, q[:rows], hist, bt[0], 0.05, acc[0])
        out = kvq.kvq_decode_step_accum_int8kv(cache, k[:1], v[:1], q[:1], bt, dev(np.array([n + 1], np.int32)), n + 1, 0.05, acc,
                                               slot_pos=sp, pos=dev(np.array([n], np.int32)))
        for budget in (n - 20, keep):  # moves in the select kernel, and page by page
            length = dev(np.array([n + 1 if budget != keep else n - 20], np.int32))
            kvq.kvq_cache_evict(cache, bt, length, n + 1, budget, acc, sp, n_sink=4, n_recent=32)
        res.append([t.cpu() for t in (out, acc, sp)] + [t[first:].cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)])
    assert kvq.kvq_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*res))
