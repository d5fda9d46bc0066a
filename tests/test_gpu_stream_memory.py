"""Calls on a stream that is not the current one, with no workspace and no outputs given: the memory they take is
that stream's, so neither what the current stream still has to do nor what it allocates next can touch it."""
import numpy as np
import pytest

import forget_ref as R
from test_gpu_evict import dev, table_of
from test_gpu_step_accum import bf

pytestmark = pytest.mark.gpu

HKV, G, D, N = 2, 4, 128, 2000


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    k.kvq_device_status()
    return k


class Side:
    """Inputs of every call, equal for equal seeds; a call changes its own side alone."""

    def __init__(self, kvq):
        import torch
        rng = np.random.default_rng(5)
        table, nb = table_of(rng, [N, N])
        self.cache = R.Pool.random(rng, nb, HKV, D).to_gpu(kvq)
        self.bt, self.lens = dev(table), dev(np.array([N, N - 100], np.int32))
        self.q, self.q4 = bf(rng, 2, HKV * G, D)[1], bf(rng, 2, 4, HKV * G, D)[1]
        self.k, self.v = bf(rng, 2, HKV, D)[1], bf(rng, 2, HKV, D)[1]
        self.qc, self.kc, self.vc = (bf(rng, 300, h, D)[1] for h in (HKV * G, HKV, HKV))
        slots = table.shape[1] * 16
        self.acc = dev(np.exp(rng.standard_normal((2, HKV, slots))).astype(np.float32))
        self.sp = torch.arange(slots, dtype=torch.int32, device="cuda").repeat(2, HKV, 1)
        self.seq, self.pos = torch.zeros(300, dtype=torch.int32, device="cuda"), torch.arange(300, dtype=torch.int32, device="cuda")
        self.first = self.lens - 1
        self.cs = dev(rng.standard_normal((400, D)).astype(np.float32))
        self.cells, self.offs = self.pos.clone(), dev(np.arange(0, 301, 30).astype(np.int32))
        self.phases = kvq.kvq_rope_phases(D)[0]

    def state(self):
        return [self.acc, self.sp, self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale]


CALLS = {
    "decode": lambda k, s, **kw: k.kvq_attn_decode_int8kv(s.cache, s.q, s.bt, s.lens, N, 0.09, **kw),
    "verify": lambda k, s, **kw: k.kvq_attn_verify_int8kv(s.cache, s.q4, s.bt, s.lens, N, 0.09, **kw),
    "step": lambda k, s, **kw: k.kvq_decode_step_int8kv(s.cache, s.k, s.v, s.q, s.bt, s.lens, N, 0.09, **kw),
    "step_accum": lambda k, s, **kw: k.kvq_decode_step_accum_int8kv(
        s.cache, s.k, s.v, s.q, s.bt, s.lens, N, 0.09, s.acc, slot_pos=s.sp, pos=s.first, **kw),
    "chunk_weights": lambda k, s, **kw: k.kvq_attn_chunk_weights_int8kv(s.cache, s.qc, N - 300, s.bt[0], 0.09, s.acc[0], **kw),
    "evict": lambda k, s, **kw: k.kvq_cache_evict(s.cache, s.bt, s.lens, N, 900, s.acc, s.sp, n_sink=4, n_recent=32, **kw),
    "rope": lambda k, s, **kw: k.kvq_rope_bf16(s.qc, s.kc, s.pos, s.phases, **kw),
    "rope_quant_write": lambda k, s, **kw: k.kvq_rope_quant_write(s.cache, s.qc, s.kc, s.vc, s.seq, s.pos, s.bt, s.cs, D, **kw),
    "prefill": lambda k, s, **kw: k.kvq_attn_prefill_int8(s.cache, s.qc, N - 300, s.bt[0], 0.09, **kw),
    "prefill_first": lambda k, s, **kw: k.kvq_attn_prefill_first_bf16(s.cache, s.qc, s.kc, s.vc, s.bt[0], 0.09, **kw),
    "sparse": lambda k, s, **kw: k.kvq_attn_sparse_int8kv(s.cache, s.qc[:10], s.offs, s.cells, s.bt[0], 0.09, **kw),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_another_stream(kvq, monkeypatch, name):
    import torch
    call, here, there = CALLS[name], Side(kvq), Side(kvq)
    want = call(kvq, here)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        if t.is_cuda:
            made.append((torch.cuda.current_stream(), t.nbytes))
        return t

    with monkeypatch.context() as m:  # who owns what the call allocates
        m.setattr(torch, "empty", spy)
        got = call(kvq, Side(kvq), stream=s)
    torch.cuda.synchronize()
    assert made and all(owner == s for owner, _ in made)
    sizes = [n for _, n in made]
    del got
    # the current stream has blocks of these sizes that it gave up with work on them outstanding, and fills
    # others as soon as the call has returned, while the call's stream has not begun
    torch.cuda._sleep(20_000_000)
    for _ in range(2):
        old = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    del old
    with torch.cuda.stream(s):
        torch.cuda._sleep(60_000_000)
    got = call(kvq, there, stream=s)
    for _ in range(2):
        old = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert kvq.kvq_device_status() == 0
    flat = lambda r: [t for t in (r if isinstance(r, tuple) else (r,))]  # noqa: E731
    for a, b in zip(flat(want) + here.state(), flat(got) + there.state()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_stream_known_by_its_handle(kvq):
    """An object of another library that has a cuda_stream, and nothing else of torch's streams."""
    import torch

    class Handle:
        pass

    s, h = torch.cuda.Stream(), Handle()
    h.cuda_stream = s.cuda_stream
    here, there = Side(kvq), Side(kvq)
    want = CALLS["evict"](kvq, here)
    torch.cuda.synchronize()
    got = CALLS["evict"](kvq, there, stream=h)
    torch.cuda.synchronize()
    assert kvq.kvq_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(list(want) + here.state(), list(got) + there.state()))
