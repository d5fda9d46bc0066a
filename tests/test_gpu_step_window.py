"""kvq_decode_step_window_int8kv against fp64: windows and first tokens that end inside pages, lengths from nothing to
past the window, verify rows, both routes; the new tokens' codes to the bit; pages that no row sees are not read;
whatever stands in masked places; refusals that only the device can see; graphs, streams, far pages."""
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


def check(pool, table, lens, cap, q, out, hkv, scale, window, sink):
    B, nq, Hq, D = q.shape
    G = Hq // hkv
    for b in range(B):
        n = max(0, min(int(lens[b]), cap))
        k, v, ok = pool.rows(table[b], n)
        for h in range(hkv):
            rows = q[b, :, h * G:(h + 1) * G].reshape(nq * G, D).astype(np.float64)
            pos = np.repeat(n - nq + np.arange(nq), G)
            o, rel, mag = WR.attend(k[h], v[h], ok, rows, pos, window, sink, scale)
            got = out[b, :, h * G:(h + 1) * G].reshape(nq * G, D)
            # a weight goes in as two fp16 parts (2^-22), O is summed over the keys and the splits
            assert (np.abs(got - o) <= (rel[:, None] + 2.0 ** -22 + n * 2.0 ** -24) * mag + 1e-30).all(), (b, h)


def run(kvq, rng, lens, hq, hkv, d, new, window, sink, write=True, split_rows=0, force=0, fill=-1, flags=0, max_ctx=None, edit=None):
    import torch
    lens = np.asarray(lens, np.int32)
    B = len(lens)
    cap = int(max(1, lens.max())) if max_ctx is None else max_ctx
    table, nb = table_of(rng, lens, spare=1)
    pool = R.Pool.random(rng, nb, hkv, d)
    if edit:
        edit(pool, table)
    # (a length past the bound is clamped to it, and the window goes by that)
    seen = WR.unread_pages(table, np.minimum(lens, cap), new, window, sink, fill)
    (q, qt), (_, kt), (_, vt) = bf(rng, B, new, hq, d), bf(rng, B, new, hkv, d), bf(rng, B, new, hkv, d)
    cache, other = pool.to_gpu(kvq), pool.to_gpu(kvq)
    scale, bt, ln = 1.0 / np.sqrt(d), dev(seen), dev(lens)
    out = torch.full((B, new, hq, d), 7.0, device="cuda")
    kvq.kvq_decode_step_window_int8kv(cache, kt if write else None, vt if write else None, qt, bt, ln, cap, scale, window, sink,
                                      out=out, split_rows=split_rows, force_route=force)
    assert kvq.kvq_device_status() == flags
    if write:  # the same codes and scales as the plain step's, and nothing else
        kvq.kvq_decode_step_int8kv(other, kt, vt, qt, dev(table), ln, cap, scale)
        kvq.kvq_device_status()
    after = R.Pool.of(cache)
    assert after.same(R.Pool.of(other))
    check(after, seen, lens, min(cap, 16 * table.shape[1]), q, out.cpu().numpy(), hkv, scale, window, sink)
    return out


WINDOWS = [(1, 0), (16, 0), (17, 4), (100, 1), (128, 16), (333, 17), (1024, 100), (5000, 4)]


@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("hq,hkv,d,new", [(24, 4, 256, 1), (8, 2, 128, 1), (8, 8, 128, 3), (24, 4, 256, 5), (16, 1, 128, 1),
                                          (6, 1, 256, 8)])
def test_windows(kvq, window, sink, hq, hkv, d, new):
    rng = np.random.default_rng(window * 31 + sink + d + new)
    lens = [2000, new, new + 1, 16, 130, 1999, window + sink + new, max(new, window - 3), 1025]
    run(kvq, rng, [n for n in lens if n <= 4000], hq, hkv, d, new, window, sink)


@pytest.mark.parametrize("force,split_rows", [(1, 0), (2, 0), (2, 16), (2, 48), (2, 512)])
@pytest.mark.parametrize("hq,hkv,d,new", [(24, 4, 256, 1), (8, 2, 128, 4)])
def test_routes(kvq, force, split_rows, hq, hkv, d, new):
    for window, sink in ((100, 40), (700, 0)):
        rng = np.random.default_rng(window + split_rows)
        run(kvq, rng, [1500, 777, 40, 128], hq, hkv, d, new, window, sink, force=force, split_rows=split_rows)
        run(kvq, rng, [1500, 777, 40, 128], hq, hkv, d, new, window, sink, write=False, force=force, split_rows=split_rows)


@pytest.mark.parametrize("G,new", [(1, 1), (9, 1), (16, 3), (4, 12), (2, 24), (3, 16), (7, 5)])
def test_groups_and_rows(kvq, G, new):
    rng = np.random.default_rng(G * 100 + new)
    for d in (128, 256):
        run(kvq, rng, [600, 333, 64], 2 * G, 2, d, new, 200, 20)


def test_lengths_that_are_not_what_they_should_be(kvq):
    """Empty sequences, fewer keys than new tokens, more than the bound, more than the table maps."""
    rng = np.random.default_rng(3)
    run(kvq, rng, [0, 300, 0], 8, 2, 128, 1, 50, 4, write=False)
    run(kvq, rng, [0, 300, 2], 8, 2, 128, 3, 50, 4, write=False)
    run(kvq, rng, [2, 300, 0], 8, 2, 128, 3, 50, 4, flags=kvq.kvq.DEV_BAD_POS)
    run(kvq, rng, [900, 300], 8, 2, 128, 1, 50, 4, max_ctx=500, write=False, flags=kvq.kvq.DEV_BAD_POS)
    run(kvq, rng, [0, 0], 8, 2, 128, 1, 50, 4, max_ctx=0, write=False)


@pytest.mark.parametrize("hq,hkv,d,new", [(24, 4, 256, 1), (8, 2, 128, 2)])
def test_a_window_of_all_is_the_plain_step(kvq, hq, hkv, d, new):
    import torch
    rng = np.random.default_rng(4)
    lens = np.array([700, 33, 1200], np.int32)
    table, nb = table_of(rng, lens)
    pool = R.Pool.random(rng, nb, hkv, d)
    a, b = pool.to_gpu(kvq), pool.to_gpu(kvq)
    qt, kt, vt = (bf(rng, 3, new, h, d)[1] for h in (hq, hkv, hkv))
    want = kvq.kvq_decode_step_int8kv(a, kt, vt, qt, dev(table), dev(lens), 1200, 0.1, force_route=2)
    for window, sink in ((1200, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 1200)):
        got = kvq.kvq_decode_step_window_int8kv(b, kt, vt, qt, dev(table), dev(lens), 1200, 0.1, window, sink, force_route=2)
        # (a plan for more keys than there are may split otherwise)
        assert torch.equal(got, want) or (got - want).abs().max() <= 1e-5 * want.abs().max()
    assert R.Pool.of(a).same(R.Pool.of(b)) and kvq.kvq_device_status() == 0


def test_pages_outside(kvq):
    """Entries that no row sees may be anything; a bad page inside is skipped and reported."""
    rng = np.random.default_rng(5)
    for fill in (-1, 2 ** 31 - 1, -2 ** 31):
        run(kvq, rng, [1500, 900], 24, 4, 256, 2, 130, 20, fill=fill)
    for page in (0, 80, 93):  # a first token's, the window's first and last

        def edit(pool, table):
            table[0, page] = -5

        run(kvq, rng, [1500, 900], 8, 2, 128, 2, 220, 20, edit=edit, write=page != 93, flags=kvq.kvq.DEV_BAD_BLOCK)


@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("d", [128, 256])
def test_masked_places_hold_anything(kvq, d, new):
    """Keys behind the window that share a page with visible ones: scales of infinity, NaN, zero and the lowest value."""
    n, window, sink = 1000, 300, 5

    def edit(pool, table):
        junk = [np.inf, -np.inf, np.nan, 0.0, np.finfo(np.float32).min, np.finfo(np.float32).max]
        low = n - new - window + 1
        for i, t in enumerate(list(range(sink, 16)) + list(range(low // 16 * 16, low))):
            page, at = table[0, t // 16], t % 16
            pool.ks[page, :, at] = junk[i % 6]
            pool.vs[page, :, at] = junk[(i + 1) % 6]
        page, at = table[0, n // 16], n % 16  # behind the sequence's end, in its last page
        pool.ks[page, :, at:], pool.vs[page, :, at:] = np.nan, np.inf

    import torch
    for force in (1, 2):
        rng = np.random.default_rng(6)
        hq, hkv = 8, 2
        table, nb = table_of(rng, [n])
        pool = R.Pool.random(rng, nb, hkv, d)
        clean = pool.copy()
        edit(pool, table)
        q = bf(rng, 1, new, hq, d)[1]
        got, want = (kvq.kvq_decode_step_window_int8kv(p.to_gpu(kvq), None, None, q, dev(table), dev(np.array([n], np.int32)), n, 0.1,
                                                       window, sink, force_route=force) for p in (pool, clean))
        # verify rows see keys one after the other: what is masked for one row may be seen by another, so only the
        # first row's window bounds what was edited
        assert torch.isfinite(got).all() and torch.equal(got, want)


def test_rows_that_are_not_finite(kvq):
    """A query row with NaN gives NaN in its own outputs alone."""
    import torch
    rng = np.random.default_rng(7)
    table, nb = table_of(rng, [500])
    pool = R.Pool.random(rng, nb, 2, 128)
    q = bf(rng, 1, 3, 8, 128)[1]
    lens = dev(np.array([500], np.int32))
    want = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), None, None, q, dev(table), lens, 500, 0.1, 100, 4)
    q[0, 1, 3, 7] = float("nan")
    got = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), None, None, q, dev(table), lens, 500, 0.1, 100, 4)
    keep = torch.ones((3, 8), dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.equal(got[0][keep], want[0][keep])


@pytest.mark.parametrize("batch,hkv,d,window", [(20, 8, 128, 1500), (11, 4, 256, 2000), (3, 2, 128, 2100), (70, 8, 128, 300)])
def test_automatic_splits(kvq, batch, hkv, d, window):
    rng = np.random.default_rng(batch)
    lens = rng.integers(window // 2, window + 700, batch)
    lens[0], lens[1] = window + 700, 1
    run(kvq, rng, lens, 2 * hkv, hkv, d, 1, window, 4)


def test_many_sequences(kvq):
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 700, 200)
    run(kvq, rng, lens, 8, 4, 128, 1, 150, 4)


def test_far_pages(kvq):
    """Codes past 2 GB and past 4 GB of the pool."""
    import torch
    rng = np.random.default_rng(9)
    hkv, d, nb = 8, 256, 140000
    cache = kvq.KVCache(nb, hkv, d)
    n, window, sink = 200, 60, 17
    table = np.full((1, 13), -1, np.int32)
    table[0, [0, 1, 8, 9, 10, 11, 12]] = [nb - 1, 70001, 139990, 5, 80000, 120000, 65536]
    small = np.full((1, 13), -1, np.int32)
    small[0, [0, 1, 8, 9, 10, 11, 12]] = np.arange(7)
    pool = R.Pool.random(rng, 7, hkv, d)
    for i, page in zip(small[0], table[0]):
        if page >= 0:
            cache.k[page], cache.v[page] = dev(pool.k[i]), dev(pool.v[i])
            cache.k_scale[page], cache.v_scale[page] = dev(pool.ks[i]), dev(pool.vs[i])
    qt, kt, vt = (bf(rng, 1, 1, h, d)[1] for h in (16, hkv, hkv))
    lens = dev(np.array([n], np.int32))
    got = kvq.kvq_decode_step_window_int8kv(cache, kt, vt, qt, dev(table), lens, n, 0.1, window, sink)
    want = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), kt, vt, qt, dev(small), lens, n, 0.1, window, sink)
    assert torch.equal(got, want) and kvq.kvq_device_status() == 0


def test_capture_and_two_streams(kvq):
    """Replayed with new lengths; two calls at once, a workspace each; the same bits every time."""
    import torch
    rng = np.random.default_rng(10)
    lens = np.array([3000, 1000], np.int32)
    table, nb = table_of(rng, lens)
    pool = R.Pool.random(rng, nb, 4, 256)
    caches = [pool.to_gpu(kvq) for _ in range(3)]
    qt, kt, vt = (bf(rng, 2, 1, h, 256)[1] for h in (24, 4, 4))
    bt, ln = dev(table), dev(lens - 5)
    need = kvq.kvq_step_window_workspace_bytes(2, 1, 24, 4, 3000, 1024, 4, 256)
    ws = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in range(3)]
    call = lambda i, **kw: kvq.kvq_decode_step_window_int8kv(caches[i], kt, vt, qt, bt, ln, 3000, 0.06, 1024, 4, workspace=ws[i], **kw)  # noqa: E731
    out = call(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, out=out)
    ln += 3
    graph.replay()
    call(1, out=torch.empty_like(out))
    ln.copy_(dev(lens - 5))
    call(1), call(2)
    ln += 3
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(out), torch.empty_like(out)]
    for _ in range(20):
        call(1, out=outs[0], stream=a)
        call(2, out=outs[1], stream=b)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], out) and kvq.kvq_device_status() == 0


def test_zero_copy(kvq):
    """Inputs and the result in mapped page-locked memory."""
    import torch
    rng = np.random.default_rng(11)
    table, nb = table_of(rng, [900])
    pool = R.Pool.random(rng, nb, 4, 256)
    qt, kt, vt = (bf(rng, 1, 1, h, 256)[1] for h in (24, 4, 4))
    lens = dev(np.array([900], np.int32))
    want = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), kt, vt, qt, dev(table), lens, 900, 0.06, 256, 4)
    host = [t.cpu().pin_memory() for t in (kt, vt, qt)]
    got = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), *host, dev(table), lens, 900, 0.06, 256, 4)
    torch.cuda.synchronize()
    assert got.device.type == "cpu" and torch.equal(got, want.cpu())


def test_a_copy_that_never_lands(kvq):
    """The bounded wait gives up: zeros or the other ranges' share, a flag, and a library that goes on working."""
    rng = np.random.default_rng(12)
    try:
        kvq.kvq_debug_fault_inject(1, 2_000_000)
        table, nb = table_of(rng, [900])
        pool = R.Pool.random(rng, nb, 4, 256)
        q = bf(rng, 1, 1, 24, 256)[1]
        out = kvq.kvq_decode_step_window_int8kv(pool.to_gpu(kvq), None, None, q, dev(table), dev(np.array([900], np.int32)), 900, 0.06,
                                                600, 4, force_route=1)
        assert kvq.kvq_device_status() == kvq.kvq.DEV_TIMEOUT
        assert bool((out[0, 0, :6] == 0).all())  # the KV head whose copy is missing
    finally:
        kvq.kvq_debug_fault_inject(0, 0)
    run(kvq, rng, [900], 24, 4, 256, 1, 600, 4)
