"""The calls around windowed attention on a stream that is not the current one, with no workspace and no outputs given: what
they allocate is that stream's (the test of the other calls, with these)."""
import pytest

import test_gpu_stream_memory as M

pytestmark = pytest.mark.gpu
kvq = M.kvq


def plan(k, s):
    return k.RopeAxes(s.phases, bytes([0, 1] * (M.D // 4)))


CALLS = {
    "step_window": lambda k, s, **kw: k.kvq_decode_step_window_int8kv(s.cache, s.k, s.v, s.q, s.bt, s.lens, M.N, 0.09, 1500, 4, **kw),
    "verify_window": lambda k, s, **kw: k.kvq_decode_step_window_int8kv(s.cache, None, None, s.q4, s.bt, s.lens, M.N, 0.09, 1500, 4, **kw),
    "prompt_window": lambda k, s, **kw: k.kvq_attn_prefill_window_int8kv(s.cache, s.qc, M.N - 300, s.bt[0], 0.09, 500, 4, **kw),
    "axes": lambda k, s, **kw: k.kvq_rope_axes_bf16(s.qc, s.kc, s.pos2, plan(k, s), **kw),
    "append": lambda k, s, **kw: k.kvq_rope_append_int8kv(s.cache, s.qc, s.kc, s.vc, s.pos2, plan(k, s), s.seq, s.pos, s.bt, **kw),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_another_stream(kvq, monkeypatch, name):
    init = M.Side.__init__

    def with_positions(self, k):
        init(self, k)
        self.pos2 = self.pos.repeat(2, 1)

    monkeypatch.setattr(M.Side, "__init__", with_positions)
    monkeypatch.setitem(M.CALLS, name, CALLS[name])
    M.test_memory_of_a_call_on_another_stream(kvq, monkeypatch, name)
