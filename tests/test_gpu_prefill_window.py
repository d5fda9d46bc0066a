"""kvq_attn_prefill_window_int8kv against fp64: chunks from one query to thousands, windows and first tokens that end
inside pages and tiles, histories from nothing on; pages that no query sees; whatever stands in masked places; the same bits
every time; a wait that runs out; and the operators together, as a serving program runs them."""
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


def run(kvq, rng, T, history, hq, hkv, d, window, sink, fill=-1, flags=0, edit=None, scale=None, out_dtype=None):
    import torch
    table, nb = table_of(rng, [history + T], spare=1)
    pool = R.Pool.random(rng, nb, hkv, d)
    if edit:
        edit(pool, table)
    seen = WR.unread_pages(table, [history + T], T, window, sink, fill)[0]
    q, qt = bf(rng, T, hq, d)
    cache, scale = pool.to_gpu(kvq), scale or 1.0 / np.sqrt(d)
    ref, tol = WR.prompt(pool, seen, q.astype(np.float64), history, window, sink, scale)
    outs = []
    for dtype in (torch.float32, torch.bfloat16):
        # rows and columns around the output are left as they were
        wide = torch.full((T + 2, hq, d), 7.0, dtype=dtype, device="cuda")
        kvq.kvq_attn_prefill_window_int8kv(cache, qt, history, dev(seen), scale, window, sink, out=wide[1:-1])
        assert kvq.kvq_device_status() == flags
        assert bool((wide[0] == 7).all()) and bool((wide[-1] == 7).all())
        got = wide[1:-1].float().cpu().numpy()
        # bf16 rounds by half a step, 2^-8 relative
        err, most = np.abs(got - ref), tol if dtype is torch.float32 else tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
        assert (err <= most).all(), (dtype, np.argwhere(err > most)[:5], (err / most).max())
        outs.append(wide[1:-1])
    return outs


@pytest.mark.parametrize("window,sink", [(1, 0), (16, 0), (100, 1), (128, 0), (129, 128), (333, 200), (1024, 4), (10000, 0), (1, 5000)])
@pytest.mark.parametrize("T,history,hq,hkv,d", [(1, 0, 4, 2, 128), (7, 5, 6, 1, 256), (33, 2000, 24, 4, 256), (130, 333, 8, 8, 128),
                                                (300, 0, 12, 2, 128), (500, 1111, 6, 2, 256)])
def test_windows(kvq, T, history, hq, hkv, d, window, sink):
    run(kvq, np.random.default_rng(T + window * 3 + sink), T, history, hq, hkv, d, window, sink)


@pytest.mark.parametrize("T,history,hq,hkv,d,window,sink", [
    (1, 4000, 24, 4, 256, 1024, 4), (1, 1, 1, 1, 128, 1, 0), (2, 129, 128, 1, 128, 50, 3), (128, 0, 1, 1, 256, 64, 0),
    (129, 127, 1, 1, 128, 127, 1), (1200, 0, 2, 2, 256, 200, 0), (5000, 0, 1, 1, 128, 300, 4), (2047, 333, 4, 1, 128, 1024, 0),
    (300, 333, 32, 8, 128, 100, 0), (500, 100, 8, 8, 128, 150, 4), (260, 500, 24, 8, 256, 60, 130), (700, 0, 10, 5, 256, 130, 1),
    (2047, 333, 16, 8, 128, 300, 0), (64, 9000, 20, 2, 256, 6000, 300), (3, 20000, 8, 1, 128, 16000, 0), (900, 100, 7, 7, 128, 77, 9), (40, 600, 48, 1, 256, 256, 16)])
def test_shapes(kvq, T, history, hq, hkv, d, window, sink):
    run(kvq, np.random.default_rng(T), T, history, hq, hkv, d, window, sink)


def test_sharp_and_flat_rows(kvq):
    """Softmax scales that leave one key, or all keys alike; V scales 2^40 apart."""
    rng = np.random.default_rng(1)
    run(kvq, rng, 200, 700, 8, 2, 128, 300, 20, scale=1e-6)

    def edit(pool, table):
        pool.vs[:] = 2.0 ** rng.integers(-30, 11, pool.vs.shape)

    for d in (128, 256):
        run(kvq, rng, 200, 700, 8, 2, d, 300, 20, edit=edit)
        run(kvq, rng, 200, 700, 8, 2, d, 300, 20, edit=edit, scale=0.5)  # weights over some 200 octaves

    def zeros(pool, table):
        pool.vs[:, :, ::2], pool.v[:, :, :, ::2] = 0.0, 0
        pool.ks[:, :, 1::4], pool.k[:, :, :, 1::4] = 0.0, 0

    run(kvq, rng, 150, 300, 8, 2, 128, 200, 5, edit=zeros)


def test_pages_outside(kvq):
    """Entries that no query sees may be anything, inside a tile that is read too; a bad page that some see is skipped."""
    rng = np.random.default_rng(2)
    for fill in (-1, 2 ** 31 - 1, -2 ** 31):
        run(kvq, rng, 100, 1500, 8, 2, 128, 130, 20, fill=fill)
    for page in (0, 93, 99):

        def edit(pool, table):
            table[0, page] = -5

        run(kvq, rng, 100, 1500, 8, 2, 256, 130, 20, edit=edit, flags=kvq.kvq.DEV_BAD_BLOCK)

    def all_bad(pool, table):
        table[0] = -1

    outs = run(kvq, rng, 20, 100, 8, 2, 128, 50, 0, edit=all_bad, flags=kvq.kvq.DEV_BAD_BLOCK)
    assert bool((outs[0] == 0).all())  # rows that see no key


def test_masked_places_hold_anything(kvq):
    """Hidden keys in pages and tiles that are read: scales of infinity, NaN, zero and the lowest value."""
    import torch
    T, history, window, sink, hq, hkv, d = 1, 1003, 300, 5, 8, 2, 128
    rng = np.random.default_rng(3)
    table, nb = table_of(rng, [1024])
    pool = R.Pool.random(rng, nb, hkv, d)
    q = bf(rng, T, hq, d)[1]
    junk = [np.inf, -np.inf, np.nan, 0.0, np.finfo(np.float32).min, np.finfo(np.float32).max]
    dirty = pool.copy()
    low = history - window + 1
    for i, t in enumerate(list(range(sink, 128)) + list(range(low // 128 * 128, low)) + list(range(history + T, 1024))):
        page, at = table[0, t // 16], t % 16
        dirty.ks[page, :, at] = junk[i % 6]
        dirty.vs[page, :, at] = junk[(i + 1) % 6]
    got, want = (kvq.kvq_attn_prefill_window_int8kv(p.to_gpu(kvq), q, history, dev(table[0]), 0.1, window, sink) for p in (dirty, pool))
    assert torch.isfinite(got).all() and torch.equal(got, want)
    # causal: what a later key holds does not reach the queries before it (all of them see the same tile)
    T = 60
    q = bf(rng, T, hq, d)[1]
    dirty = pool.copy()
    last = 903 + T - 1
    dirty.vs[table[0, last // 16], :, last % 16] = np.nan
    got, want = (kvq.kvq_attn_prefill_window_int8kv(p.to_gpu(kvq), q, 903, dev(table[0]), 0.1, window, sink) for p in (dirty, pool))
    assert torch.equal(got[:-1], want[:-1]) and torch.isnan(got[-1].float()).all()


def test_rows_that_are_not_finite(kvq):
    import torch
    rng = np.random.default_rng(4)
    table, nb = table_of(rng, [700])
    pool = R.Pool.random(rng, nb, 2, 256)
    q = bf(rng, 100, 8, 256)[1]
    call = lambda: kvq.kvq_attn_prefill_window_int8kv(pool.to_gpu(kvq), q, 600, dev(table[0]), 0.06, 150, 4)  # noqa: E731
    want = call()
    q[17, 3, 5], q[50, 0, 9] = float("nan"), float("inf")
    got = call()
    keep = torch.ones((100, 8), dtype=torch.bool, device="cuda")
    keep[17, 3] = keep[50, 0] = False
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[17, 3].float()).all()


def test_the_same_bits(kvq):
    """Twice, replayed from a graph with other inputs, and two calls at once with a workspace each."""
    import torch
    rng = np.random.default_rng(5)
    table, nb = table_of(rng, [3000])
    pool = R.Pool.random(rng, nb, 4, 256)
    cache, row = pool.to_gpu(kvq), dev(table[0])
    q, other = bf(rng, 400, 24, 256)[1], bf(rng, 400, 24, 256)[1]
    need = kvq.kvq_prefill_window_workspace_bytes(400, 24, 4, 2600, 1024, 4, 256)
    ws = [torch.full((need,), v, dtype=torch.uint8, device="cuda") for v in (0, 255, 127)]
    call = lambda i, x, **kw: kvq.kvq_attn_prefill_window_int8kv(cache, x, 2600, row, 0.06, 1024, 4, workspace=ws[i], **kw)  # noqa: E731
    a, b = call(0, q), call(1, q)
    assert torch.equal(a, b)
    x, out = q.clone(), torch.empty_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(2, x, out=out)
    x.copy_(other)
    graph.replay()
    c = call(0, other)
    assert torch.equal(out, c)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = torch.empty_like(a), torch.empty_like(a)
    torch.cuda.synchronize()
    for _ in range(10):
        call(0, q, out=o1, stream=s)
        call(1, other, out=o2, stream=t)
    torch.cuda.synchronize()
    assert torch.equal(o1, a) and torch.equal(o2, c) and kvq.kvq_device_status() == 0


def test_a_copy_that_never_lands(kvq):
    import torch
    rng = np.random.default_rng(6)
    table, nb = table_of(rng, [2000])
    pool = R.Pool.random(rng, nb, 2, 128)
    q = bf(rng, 500, 8, 128)[1]
    cache, row = pool.to_gpu(kvq), dev(table[0])
    want = kvq.kvq_attn_prefill_window_int8kv(cache, q, 1500, row, 0.09, 600, 4)
    out = torch.full_like(want, 7.0)
    try:
        kvq.kvq_debug_fault_inject(5, 20_000_000)
        kvq.kvq_attn_prefill_window_int8kv(cache, q, 1500, row, 0.09, 600, 4, out=out)
        assert kvq.kvq_device_status() == kvq.kvq.DEV_TIMEOUT
    finally:
        kvq.kvq_debug_fault_inject(0, 0)
    left = (out == 7.0).all(-1)
    assert bool(left[0, 0]) and bool((left | (out == want).all(-1)).all())  # each row as it was, or right
    assert not bool(left.all())
    got = kvq.kvq_attn_prefill_window_int8kv(cache, q, 1500, row, 0.09, 600, 4)
    assert torch.equal(got, want) and kvq.kvq_device_status() == 0


def test_far_pages(kvq):
    import torch
    rng = np.random.default_rng(7)
    hkv, d, nb, n = 8, 256, 140000, 200
    cache = kvq.KVCache(nb, hkv, d)
    table = np.array([139999, 70001, 3, 139990, 5, 80000, 120000, 65536, 131072, 99999, 1, 100000, 131073], np.int32)
    pool = R.Pool.random(rng, 13, hkv, d)
    for i, page in enumerate(table):
        cache.k[page], cache.v[page] = dev(pool.k[i]), dev(pool.v[i])
        cache.k_scale[page], cache.v_scale[page] = dev(pool.ks[i]), dev(pool.vs[i])
    q = bf(rng, 50, 16, d)[1]
    got = kvq.kvq_attn_prefill_window_int8kv(cache, q, n - 50, dev(table), 0.06, 90, 17)
    want = kvq.kvq_attn_prefill_window_int8kv(pool.to_gpu(kvq), q, n - 50, dev(np.arange(13, dtype=np.int32)), 0.06, 90, 17)
    assert torch.equal(got, want) and kvq.kvq_device_status() == 0


@pytest.mark.parametrize("hq,hkv,d,sections", [(24, 4, 256, [48, 40, 40]), (8, 2, 128, [24, 20, 20])])
def test_a_prompt_and_its_answer(kvq, hq, hkv, d, sections):
    """Two prompt chunks with positions on three axes, then new tokens one by one: each chunk is rotated and appended and
    attends; each new token is rotated (its k not appended) and written by the step.  Against 64 bits from the codes in the cache."""
    import torch
    rng = np.random.default_rng(d)
    window, sink, scale = 150, 20, 1.0 / np.sqrt(d)
    plan = kvq.kvq_rope_axes_phases(sections, 1.0e6, "turns")
    table, nb = table_of(rng, [400])
    cache, bt = kvq.KVCache(nb, hkv, d), dev(table)
    at = 0
    for T in (133, 170):
        qkv = bf(rng, T, hq + 2 * hkv, d)[1]
        pos = dev(np.stack([at + np.arange(T) // 7, np.arange(T) % 7, np.arange(T) % 5]).astype(np.int32))
        slot = torch.arange(at, at + T, dtype=torch.int32, device="cuda")
        q = kvq.kvq_rope_append_int8kv(cache, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, plan, torch.zeros_like(slot), slot, bt)
        out = kvq.kvq_attn_prefill_window_int8kv(cache, q, at, bt[0], scale, window, sink, out_dtype=torch.float32)
        ref, tol = WR.prompt(R.Pool.of(cache), table[0], q.double().cpu().numpy(), at, window, sink, scale)
        assert (np.abs(out.cpu().numpy() - ref) <= tol).all()
        at += T
    for i in range(5):
        qkv = bf(rng, 1, hq + 2 * hkv, d)[1]
        pos = torch.full((3, 1), 1000 + i, dtype=torch.int32, device="cuda")
        q, k = kvq.kvq_rope_axes_bf16(qkv[:, :hq], qkv[:, hq:hq + hkv], pos, plan)
        at += 1
        lens = dev(np.array([at], np.int32))
        out = kvq.kvq_decode_step_window_int8kv(cache, k, qkv[:, hq + hkv:].contiguous(), q, bt, lens, 400, scale, window, sink)
        pool = R.Pool.of(cache)
        ref, tol = WR.prompt(pool, table[0], q.double().cpu().numpy(), at - 1, window, sink, scale)
        assert (np.abs(out.cpu().numpy() - ref) <= tol).all()
        # the same query as a chunk of one
        one = kvq.kvq_attn_prefill_window_int8kv(cache, q, at - 1, bt[0], scale, window, sink, out_dtype=torch.float32)
        assert (np.abs(one.cpu().numpy() - ref) <= tol).all()
    assert kvq.kvq_device_status() == 0
