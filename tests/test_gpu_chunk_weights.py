"""kvq_attn_chunk_weights_int8kv against fp64 softmax weights: tile edges, causal masks, GQA groups, one
token to long chunks, split runs, bad pages, non-finite rows, failures, streams and graphs."""
import numpy as np
import pytest

import forget_ref as R
from test_gpu_evict import dev, same, table_of
from test_gpu_step_accum import bf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


def check(pool, row, hist, q, acc0, acc, scale):
    T, Hq, D = q.shape
    n, G = hist + T, Hq // pool.hkv
    k, v, ok = pool.rows(row, n)
    for h in range(pool.hkv):
        rows = q[:, h * G:(h + 1) * G].reshape(T * G, D).astype(np.float64)
        p, _, rel, _ = R.weights(k[h], v[h], ok, rows, hist + 1 + np.arange(T).repeat(G), scale)
        ref = acc0[h, :n] + p.sum(0)
        # beside the weights' own errors (R.weights): 32 columns are summed in four chains (10 roundings), then two
        # such sums a tile, the parts (at most four a run) and acc: 10 + 2 tiles + parts + 1 roundings, within
        # 96 + tiles for the cases' 19 tiles and the few runs that share a key tile
        tol = (rel[:, None] * p).sum(0) + (96 + -(-T * G // 128)) * 2.0 ** -24 * np.abs(ref) + 1e-30
        bad = np.abs(acc[h, :n] - ref) > tol
        assert not bad.any(), (h, np.argwhere(bad)[:4].ravel(), np.abs(acc[h, :n] - ref).max())
        assert same(acc[h, n:], acc0[h, n:])


CASES = [  # tokens, history, hkv, G, d
    (1, 0, 1, 1, 128), (1, 0, 2, 6, 256), (2, 0, 1, 16, 256), (1, 127, 1, 4, 128), (1, 128, 2, 3, 256), (7, 121, 1, 1, 256),
    (128, 0, 1, 1, 128), (129, 0, 1, 1, 256), (22, 500, 4, 6, 256), (21, 1, 1, 6, 128), (128, 128, 2, 1, 256),
    (100, 413, 2, 4, 128), (333, 47, 1, 5, 256), (513, 0, 2, 2, 128), (64, 1999, 8, 4, 128), (40, 3000, 1, 12, 256),
    (5, 700, 3, 20, 128), (777, 600, 1, 3, 256),
    (1, 40000, 3, 1, 128), (1, 30000, 2, 1, 256), (129, 20000, 1, 1, 256), (30, 2500, 3, 8, 256), (100, 1500, 2, 5, 128),
    (3, 5, 300, 2, 128), (150, 90, 200, 1, 256), (260, 10, 170, 1, 128),  # more KV heads than SMs
    (120, 900, 2, 6, 128), (110, 900, 2, 6, 256), (150, 900, 2, 6, 128), (150, 5000, 3, 6, 256)]


@pytest.mark.parametrize("T,hist,hkv,G,d", CASES)
def test_weights(kvq, T, hist, hkv, G, d):
    rng = np.random.default_rng(T * 131 + hist + G + d)
    table, nb = table_of(rng, [hist + T], spare=3)
    pool = R.Pool.random(rng, nb, hkv, d)
    slots = table.shape[1] * 16 + 5
    q, qt = bf(rng, T, hkv * G, d)
    q[0] *= 0  # a row of zeros: uniform weights
    qt[0] = 0
    acc0 = np.exp(rng.standard_normal((hkv, slots))).astype(np.float32)
    acc = dev(acc0)
    kvq.kvq_attn_chunk_weights_int8kv(pool.to_gpu(kvq), qt, hist, dev(table[0]), 1.0 / np.sqrt(d), acc)
    assert kvq.kvq_device_status() == 0
    check(pool, table[0], hist, q, acc0, acc.cpu().numpy(), 1.0 / np.sqrt(d))


def test_rows_of_every_size(kvq):
    """Queries of very different magnitudes in one chunk (2^-60 to 2^9) and sharp softmaxes: each row is
    scaled on its own."""
    rng = np.random.default_rng(7)
    T, hist, hkv, G, d = 90, 300, 1, 2, 256
    table, nb = table_of(rng, [hist + T])
    pool = R.Pool.random(rng, nb, hkv, d)
    q, qt = bf(rng, T, G, d)
    f = 2.0 ** np.linspace(-60, 9, T).round()[:, None, None]
    q = (q * f).astype(np.float32)
    import torch
    qt = torch.from_numpy(q).to(torch.bfloat16).cuda()
    acc0 = np.zeros((hkv, 400), np.float32)
    acc = dev(acc0)
    kvq.kvq_attn_chunk_weights_int8kv(pool.to_gpu(kvq), qt, hist, dev(table[0]), 0.0625, acc)
    check(pool, table[0], hist, q, acc0, acc.cpu().numpy(), 0.0625)


def test_long_chunks_sum_to_the_rows(kvq):
    """Many tiles a run, runs that share tiles: every row gives weight 1, whichever CTAs its keys went to."""
    import torch
    rng = np.random.default_rng(8)
    for T, hist, hkv, G, d in ((2048, 5000, 2, 6, 256), (1500, 9001, 8, 4, 128), (33, 20000, 4, 4, 256)):
        table, nb = table_of(rng, [hist + T])
        cache = R.Pool.random(rng, nb, hkv, d).to_gpu(kvq)
        acc = torch.zeros((hkv, hist + T), device="cuda")
        kvq.kvq_attn_chunk_weights_int8kv(cache, bf(rng, T, hkv * G, d)[1], hist, dev(table[0]), 0.06, acc)
        s = acc.double().sum(1).cpu().numpy()
        # l and the weights carry the same scores up to their roundings (1e-5 relative at these sizes), sums of
        # 64 columns and of the tiles round a few hundred times in all
        assert np.abs(s - T * G).max() <= T * G * (1e-5 + 500 * 2.0 ** -24), s
    assert kvq.kvq_device_status() == 0


def test_agrees_with_the_decode_step(kvq):
    """A chunk of two queries is a verify step of two rows."""
    import torch
    rng = np.random.default_rng(9)
    n, hkv, G, d = 900, 2, 6, 256
    table, nb = table_of(rng, [n])
    pool = R.Pool.random(rng, nb, hkv, d)
    cache = pool.to_gpu(kvq)
    q, qt = bf(rng, 2, hkv * G, d)
    a, b = torch.zeros((hkv, n), device="cuda"), torch.zeros((1, hkv, n), device="cuda")
    kvq.kvq_attn_chunk_weights_int8kv(cache, qt, n - 2, dev(table[0]), 0.0625, a)
    kvq.kvq_decode_step_accum_int8kv(cache, None, None, qt[None], dev(table), dev(np.array([n], np.int32)), n, 0.0625, b)
    zero = np.zeros((hkv, n), np.float32)
    check(pool, table[0], n - 2, q, zero, a.cpu().numpy(), 0.0625)
    check(pool, table[0], n - 2, q, zero, b[0].cpu().numpy(), 0.0625)


def test_bad_pages_get_no_weight(kvq):
    from int8_kv_cache_quant_gb300.kvq import DEV_BAD_BLOCK
    rng = np.random.default_rng(10)
    T, hist, hkv, G, d = 60, 340, 2, 3, 128
    table, nb = table_of(rng, [hist + T])
    table[0, [0, 9, 24]] = [-1, nb, 1 << 30]
    pool = R.Pool.random(rng, nb, hkv, d)
    q, qt = bf(rng, T, hkv * G, d)
    acc0 = np.full((hkv, 400), 2.0, np.float32)
    acc = dev(acc0)
    kvq.kvq_attn_chunk_weights_int8kv(pool.to_gpu(kvq), qt, hist, dev(table[0]), 0.09, acc)
    assert kvq.kvq_device_status() == DEV_BAD_BLOCK
    check(pool, table[0], hist, q, acc0, acc.cpu().numpy(), 0.09)
    assert (acc.cpu().numpy()[:, :16] == 2).all()
    # every page bad: no row has a key, nothing is added
    acc = dev(acc0)
    kvq.kvq_attn_chunk_weights_int8kv(pool.to_gpu(kvq), qt, hist, dev(np.full_like(table[0], -5)), 0.09, acc)
    assert kvq.kvq_device_status() == DEV_BAD_BLOCK
    assert same(acc.cpu().numpy(), acc0)


def test_a_row_that_is_not_finite_reaches_only_the_keys_it_sees(kvq):
    import torch
    rng = np.random.default_rng(11)
    T, hist, hkv, G, d = 200, 60, 1, 2, 128
    table, nb = table_of(rng, [hist + T])
    pool = R.Pool.random(rng, nb, hkv, d)
    q, qt = bf(rng, T, G, d)
    qt[50, 1, 3] = float("nan")
    acc = torch.zeros((1, hist + T), device="cuda")
    kvq.kvq_attn_chunk_weights_int8kv(pool.to_gpu(kvq), qt, hist, dev(table[0]), 0.09, acc)
    a = acc.cpu().numpy()[0]
    assert np.isnan(a[:hist + 51]).all() and np.isfinite(a[hist + 51:]).all()


def test_a_wait_that_ran_out(kvq):
    """The first run of the row pass stops at its first tile (host-injected): the call returns, the rows it
    left unfinished give no weight, and the next call is right again."""
    import torch
    from int8_kv_cache_quant_gb300.kvq import DEV_TIMEOUT
    rng = np.random.default_rng(12)
    T, hist, hkv, G, d = 64, 9000, 1, 2, 128
    table, nb = table_of(rng, [hist + T])
    pool = R.Pool.random(rng, nb, hkv, d)
    cache, bt = pool.to_gpu(kvq), dev(table[0])
    q, qt = bf(rng, 1000, G, d)
    acc = torch.zeros((1, hist + T), device="cuda")
    T2 = 1000  # several tiles a run
    table2, nb2 = table_of(rng, [T2 + 3000])
    cache2, bt2 = R.Pool.random(rng, nb2, hkv, d).to_gpu(kvq), dev(table2[0])
    acc2 = torch.zeros((1, T2 + 3000), device="cuda")
    try:
        kvq.kvq_debug_fault_inject(4, 20_000_000)
        kvq.kvq_attn_chunk_weights_int8kv(cache2, qt, 3000, bt2, 0.09, acc2)
        assert kvq.kvq_device_status() == DEV_TIMEOUT
    finally:
        kvq.kvq_debug_fault_inject(0, 0)
    s = float(acc2.double().sum())
    # the 256 rows of the first run's row tiles are gone, the others give 1 each
    assert abs(s - (T2 * G - 256)) < 0.1, s
    kvq.kvq_attn_chunk_weights_int8kv(cache, qt[:T], hist, bt, 0.09, acc)
    assert kvq.kvq_device_status() == 0
    check(pool, table[0], hist, q[:T], np.zeros((1, hist + T), np.float32), acc.cpu().numpy(), 0.09)


def test_same_bits_on_another_stream_and_in_a_graph(kvq):
    import torch
    rng = np.random.default_rng(13)
    T, hist, hkv, G, d = 70, 2500, 2, 4, 128
    table, nb = table_of(rng, [hist + T])
    cache, bt = R.Pool.random(rng, nb, hkv, d).to_gpu(kvq), dev(table[0])
    qt = bf(rng, T, hkv * G, d)[1]
    need = kvq.kvq_chunk_weights_workspace_bytes(T, hkv * G, hkv, hist, d)
    w = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    accs = [torch.zeros((hkv, hist + T), device="cuda") for _ in range(3)]
    kvq.kvq_attn_chunk_weights_int8kv(cache, qt, hist, bt, 0.09, accs[0], workspace=w[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kvq.kvq_attn_chunk_weights_int8kv(cache, qt, hist, bt, 0.09, accs[1], workspace=w[1], stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_attn_chunk_weights_int8kv(cache, qt, hist, bt, 0.09, accs[2], workspace=w[0])
    accs[2].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(accs[0], accs[1]) and torch.equal(accs[0], accs[2])
    assert kvq.kvq_device_status() == 0


def test_two_streams_at_once(kvq):
    """Calls of different shapes on two streams, each with its own workspace: the bits of calls one by one."""
    import torch
    rng = np.random.default_rng(17)
    hkv, G, d = 2, 4, 256
    table, nb = table_of(rng, [1300])
    cache, bt = R.Pool.random(rng, nb, hkv, d).to_gpu(kvq), dev(table[0])
    shapes = [(20, 900), (300, 1000), (1, 1200), (64, 0)]
    qs = [bf(rng, T, hkv * G, d)[1] for T, _ in shapes]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    size = max(kvq.kvq_chunk_weights_workspace_bytes(T, hkv * G, hkv, h, d) for T, h in shapes)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
    want = torch.zeros((4, hkv, 1301), device="cuda")
    got = torch.zeros((2, 4, hkv, 1301), device="cuda")
    for i, (T, h) in enumerate(shapes):
        for _ in range(3):
            kvq.kvq_attn_chunk_weights_int8kv(cache, qs[i], h, bt, 0.07, want[i], workspace=ws[2])
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (T, h) in enumerate(shapes):
            for s in range(2):
                j = (i + s) % 4
                kvq.kvq_attn_chunk_weights_int8kv(cache, qs[j], shapes[j][1], bt, 0.07, got[s, j], workspace=ws[s], stream=streams[s])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
    assert kvq.kvq_device_status() == 0


def test_refused_tensors(kvq):
    import torch
    c = kvq.KVCache(8, 2, 128)
    ok = dict(cache=c, q=torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda"), history_len=10,
              block_table_row=torch.zeros(8, dtype=torch.int32, device="cuda"), softmax_scale=0.1,
              acc=torch.zeros((2, 14), device="cuda"))
    for bad in (dict(q=ok["q"].float()), dict(q=ok["q"].cpu()), dict(q=ok["q"][:, :, :64]), dict(q=ok["q"][:, ::2]),
                dict(acc=ok["acc"][:, :13]), dict(acc=ok["acc"][:1]), dict(acc=ok["acc"].double()), dict(acc=ok["acc"][0]),
                dict(block_table_row=ok["block_table_row"].long())):
        with pytest.raises(ValueError):
            kvq.kvq_attn_chunk_weights_int8kv(**(ok | bad))
    for bad in (dict(softmax_scale=-1.0), dict(history_len=-1), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_attn_chunk_weights_int8kv(**(ok | bad))
