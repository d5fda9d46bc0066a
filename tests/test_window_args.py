"""Refusals and host arithmetic of the operators around windowed attention: no GPU, nothing is launched."""
import ctypes

import numpy as np
import pytest

import forget_ref as R
import int8_kv_cache_quant_gb300 as k
import window_ref as WR

A = 256  # an aligned address that is never used
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return k.lib()


def cache(d=256, hkv=4, block=16, kp=A):
    return k.kvq._Cache(kp, A, A, A, 8, block, hkv, d)


def step(L, c=None, k_new=A, v_new=A, q=A, batch=1, n_new=1, hq=24, bt=A, mb=8, ctx=A, max_ctx=100, w=50, sink=4, out=A, ws=A,
         wb=1 << 30, opts=None):
    return L.kvq_decode_step_window_int8kv(ctypes.byref(c or cache()), k_new, v_new, q, batch, n_new, hq, bt, mb, ctx, max_ctx, 0.1, w,
                                           sink, out, ws, wb, ctypes.byref(opts) if opts else None, None)


def opts(split=0, force=0):
    return k.kvq._decode_opts(split, 0, force)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(w=0)), (INVALID, dict(w=-1)), (INVALID, dict(sink=-1)), (INVALID, dict(q=None)), (INVALID, dict(out=None)),
    (INVALID, dict(ctx=None)), (INVALID, dict(bt=None)), (INVALID, dict(k_new=None)), (INVALID, dict(v_new=None)), (INVALID, dict(hq=23)),
    (INVALID, dict(batch=0)), (INVALID, dict(n_new=0)), (INVALID, dict(max_ctx=-1)), (INVALID, dict(opts=opts(split=24))),
    (INVALID, dict(opts=opts(force=3))), (UNSUPPORTED, dict(hq=4 * 17)), (UNSUPPORTED, dict(n_new=9)), (UNSUPPORTED, dict(batch=65536)),
    (UNSUPPORTED, dict(c=cache(d=192))), (UNSUPPORTED, dict(mb=1 << 27)), (UNSUPPORTED, dict(max_ctx=1 << 30, w=1 << 30, opts=opts(16, 2))),
    (MISALIGNED, dict(q=A + 2)), (MISALIGNED, dict(k_new=A + 8)), (MISALIGNED, dict(out=A + 4)), (MISALIGNED, dict(ctx=A + 1)),
    (MISALIGNED, dict(ws=A + 8, opts=opts(16, 2))), (WORKSPACE, dict(ws=None, opts=opts(16, 2))),
    (WORKSPACE, dict(wb=1000, opts=opts(16, 2)))])
def test_step_refusals(L, status, kw):
    assert step(L, **kw) == status


def test_step_workspace(L):
    # the keys that count: pages of the first tokens, and of a window that may begin at the end of a page
    need = lambda *a, **kw: k.kvq_step_window_workspace_bytes(*a, **kw)  # noqa: E731
    full = lambda keys: k.kvq_verify_workspace_bytes(2, 3, 8, keys, 128, split_rows=64)  # noqa: E731
    assert need(2, 3, 8, 2, 100000, 1000, 5, 128, split_rows=64) == full(16 + 16 * ((1000 + 2 + 30) // 16))
    assert need(2, 3, 8, 2, 500, 1000, 5, 128, split_rows=64) == full(500)
    assert need(2, 3, 8, 2, 1 << 30, 2 ** 31 - 1, 2 ** 31 - 1, 128, split_rows=65536) == k.kvq_verify_workspace_bytes(
        2, 3, 8, 1 << 30, 128, split_rows=65536)
    assert need(2, 3, 8, 2, 500, 0, 5, 128) == 0 and need(2, 3, 8, 2, 500, 5, -1, 128) == 0
    assert need(1, 1, 24, 4, 100000, 30, 0, 256) == 0  # one split: the single-CTA route
    n = need(2, 3, 8, 2, 100000, 1000, 5, 128, split_rows=64)
    kw = dict(c=cache(d=128, hkv=2), batch=2, n_new=3, hq=8, max_ctx=100000, mb=6250, w=1000, sink=5, opts=opts(split=64))
    assert step(L, wb=n - 1, **kw) == WORKSPACE


def prompt(L, c=None, q=A, n=10, hq=24, hist=20, bt=A, nb=8, scale=0.1, w=50, sink=4, out=A, kind=1, ws=A, wb=1 << 40):
    return L.kvq_attn_prefill_window_int8kv(ctypes.byref(c or cache()), q, n, hq, hist, bt, nb, scale, w, sink, out, kind, ws, wb, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(bt=None)), (INVALID, dict(out=None)), (INVALID, dict(n=0)), (INVALID, dict(hq=0)),
    (INVALID, dict(hq=26)), (INVALID, dict(hist=-1)), (INVALID, dict(nb=0)), (INVALID, dict(nb=1)), (INVALID, dict(w=0)),
    (INVALID, dict(w=-5)), (INVALID, dict(sink=-1)), (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-0.1)), (INVALID, dict(scale=NAN)),
    (INVALID, dict(scale=INF)), (UNSUPPORTED, dict(kind=2)), (UNSUPPORTED, dict(kind=-1)),
    (UNSUPPORTED, dict(c=cache(hkv=64), hq=65536)), (WORKSPACE, dict(c=cache(hkv=64), hq=65536 - 64, ws=None)),
    (UNSUPPORTED, dict(c=cache(hkv=1), hq=1025)), (WORKSPACE, dict(c=cache(hkv=1), hq=1024, ws=None)),
    (UNSUPPORTED, dict(n=1 << 28, hist=0, nb=1 << 24)), (UNSUPPORTED, dict(hist=(1 << 30) - 10, nb=1 << 27)),
    (UNSUPPORTED, dict(n=1 << 25, hist=1 << 29, nb=1 << 26)), (UNSUPPORTED, dict(c=cache(hkv=65536), hq=65536)),
    (UNSUPPORTED, dict(c=cache(d=64))), (MISALIGNED, dict(q=A + 8)), (MISALIGNED, dict(out=A + 8)), (MISALIGNED, dict(bt=A + 2)),
    (MISALIGNED, dict(ws=A + 8)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(wb=1000))])
def test_prompt_refusals(L, status, kw):
    assert prompt(L, **kw) == status


def prompt_tiles(T, hq, hkv, hist, window, sink):
    """(pairs of 128-row and 128-key tiles of a KV head that share a visible key, key tiles of them), by their definition."""
    G = hq // hkv
    pairs, tiles = 0, set()
    for r0 in range(0, T * G, 128):
        i0, i1 = r0 // G, min(r0 + 127, T * G - 1) // G
        # the tiles from the first query's window to the last query, and those of the first tokens
        mine = set(range(max(0, hist + i0 - window + 1) // 128, (hist + i1) // 128 + 1)) | set(range(min(-(-sink // 128), (hist + i1) // 128 + 1)))
        pairs += len(mine)
        tiles |= mine
    return pairs, len(tiles)


@pytest.mark.parametrize("T,hq,hkv,hist,window,sink,d", [
    (10, 24, 4, 20, 50, 4, 256), (1, 1, 1, 0, 1, 0, 128), (2048, 24, 4, 30720, 4096, 4, 256), (500, 6, 2, 1111, 129, 300, 128),
    (300, 8, 8, 5000, 77, 20000, 128), (33, 24, 4, 5000, 2 ** 31 - 1, 2 ** 31 - 1, 256)])
def test_prompt_workspace(L, T, hq, hkv, hist, window, sink, d):
    pairs, tiles = prompt_tiles(T, hq, hkv, hist, window, sink)
    runs = min(160, max(1, pairs * hkv // 2))  # of two tile pairs at least
    want = hkv * tiles * (4 * 128 * d + 1536) + runs * 2 * 128 * (d + 2) * 4
    assert k.kvq_prefill_window_workspace_bytes(T, hq, hkv, hist, window, sink, d) == want
    kw = dict(c=cache(d=d, hkv=hkv), n=T, hq=hq, hist=hist, nb=-(-(hist + T) // 16), w=window, sink=sink)
    assert prompt(L, wb=want - 1, **kw) == WORKSPACE


def test_prompt_workspace_of_nothing(L):
    need = k.kvq_prefill_window_workspace_bytes
    assert need(0, 24, 4, 20, 50, 4, 256) == need(10, 23, 4, 20, 50, 4, 256) == need(10, 24, 4, -1, 50, 4, 256) == 0
    assert need(10, 24, 4, 20, 0, 4, 256) == need(10, 24, 4, 20, 50, -1, 256) == need(10, 24, 4, 20, 50, 4, 192) == 0
    assert need(1 << 28, 24, 4, 0, 50, 4, 256) == 0


MAP = bytes([0, 1, 2] * 42 + [0, 0])


def axes(L, q=A, qo=A, qs=24 * 256, qos=24 * 256, hq=24, kk=A, ko=A, ks=1024, kos=1024, hk=4, d=256, T=10, pos=A, ps=10, n=3, ph=A,
         axis_of=MAP, r=256, off=0, layout=0, f=1.0, inv=0):
    return L.kvq_rope_axes_bf16(q, qo, qs, qos, hq, kk, ko, ks, kos, hk, d, T, pos, ps, n, ph, axis_of, r, off, layout, f, inv, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(qo=None)), (INVALID, dict(kk=None)), (INVALID, dict(pos=None)), (INVALID, dict(ph=None)),
    (INVALID, dict(axis_of=None)), (INVALID, dict(axis_of=b"\3" * 128)), (INVALID, dict(ps=9)), (INVALID, dict(T=-1)),
    (INVALID, dict(r=255)), (INVALID, dict(r=0)), (INVALID, dict(off=2)), (INVALID, dict(qs=24 * 256 - 1)), (INVALID, dict(qos=24 * 256 + 8)),
    (UNSUPPORTED, dict(n=0)), (UNSUPPORTED, dict(n=5)), (UNSUPPORTED, dict(layout=2)), (UNSUPPORTED, dict(d=1025)),
    (MISALIGNED, dict(q=A + 1)), (MISALIGNED, dict(pos=A + 2)), (MISALIGNED, dict(ph=A + 4)), (0, dict(T=0)), (0, dict(hq=0, hk=0))])
def test_axes_refusals(L, status, kw):
    assert axes(L, **kw) == status


def append(L, c=None, q=A, qo=A, qs=6144, qos=6144, hq=24, kk=A, ks=1024, v=A, vs=1024, T=10, seq=A, slot=A, bt=A, ns=2, mb=8, pos=A,
           ps=10, n=3, ph=A, axis_of=MAP, r=256, off=0, layout=0, f=1.0):
    return L.kvq_rope_append_int8kv(ctypes.byref(c or cache()), q, qo, qs, qos, hq, kk, ks, v, vs, T, seq, slot, bt, ns, mb, pos, ps, n,
                                    ph, axis_of, r, off, layout, f, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(qo=None)), (INVALID, dict(kk=None)), (INVALID, dict(v=None)), (INVALID, dict(seq=None)),
    (INVALID, dict(slot=None)), (INVALID, dict(bt=None)), (INVALID, dict(pos=None)), (INVALID, dict(ph=None)), (INVALID, dict(axis_of=None)),
    (INVALID, dict(axis_of=b"\3" * 128)), (INVALID, dict(ps=9)), (INVALID, dict(T=-1)), (INVALID, dict(hq=-1)), (INVALID, dict(ns=0)),
    (INVALID, dict(mb=0)), (INVALID, dict(r=258)), (INVALID, dict(off=8)), (INVALID, dict(ks=1016)), (INVALID, dict(vs=1016)),
    (INVALID, dict(qos=6152)), (INVALID, dict(f=NAN)), (INVALID, dict(f=INF)), (UNSUPPORTED, dict(r=24, axis_of=MAP)),
    (UNSUPPORTED, dict(r=128, off=4)), (UNSUPPORTED, dict(n=0)), (UNSUPPORTED, dict(n=5)), (UNSUPPORTED, dict(layout=2)),
    (UNSUPPORTED, dict(c=cache(d=64))), (UNSUPPORTED, dict(c=cache(block=32))), (UNSUPPORTED, dict(mb=1 << 27)),
    (UNSUPPORTED, dict(hq=65536)), (MISALIGNED, dict(q=A + 8)), (MISALIGNED, dict(kk=A + 8)), (MISALIGNED, dict(v=A + 2)),
    (MISALIGNED, dict(ks=1028)), (MISALIGNED, dict(qo=2 * A, qos=6146)), (MISALIGNED, dict(slot=A + 2)), (MISALIGNED, dict(ph=A + 4)),
    (MISALIGNED, dict(c=cache(kp=A + 4))), (0, dict(T=0))])
def test_append_refusals(L, status, kw):
    assert append(L, **kw) == status


@pytest.mark.parametrize("order", ["chunked", "turns"])
@pytest.mark.parametrize("sections", [[64], [24, 20, 20], [16, 24, 24], [1, 5], [0, 3, 0, 4], [7, 0, 0]])
@pytest.mark.parametrize("kind,kw", [("none", {}), ("linear", dict(factor=4.0)), ("yarn", dict(factor=8.0, original_len=4096.0)),
                                     ("bands", dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0))])
def test_axes_phases(L, order, sections, kind, kw):
    plan = k.kvq_rope_axes_phases(sections, 1.0e6, order, "shared", kind, device="cpu", **kw)
    axis_of = WR.sections_to_axes(sections, order)
    assert list(plan.axis_of) == axis_of and plan.rotary_dim == 2 * sum(sections) and plan.n_axes == max(axis_of) + 1
    phases, factor = k.kvq_rope_phases(2 * sum(sections), 1.0e6, kind, device="cpu", **kw)
    assert np.array_equal(plan.phases.numpy(), phases.numpy()) and plan.attn_factor == factor
    own = k.kvq_rope_axes_phases(sections, 1.0e6, order, "per_axis", kind, device="cpu", **kw)
    ref_kw = {("length" if n == "original_len" else n): v for n, v in kw.items()}
    for a, n in enumerate(sections):
        if n:
            inv, factor = R.inv_freq(2 * n, 1.0e6, kind, **ref_kw)
            turns = inv / (2 * np.pi)
            got = own.phases.numpy().view(np.uint64)[np.array(axis_of) == a].astype(np.float64) / 2.0 ** 64
            # fp64 powers and quotients, and half a step of 2^-64 turns
            np.testing.assert_allclose(got, turns - np.floor(turns), rtol=16 * 2.0 ** -53, atol=2.0 ** -65)
            assert own.attn_factor == np.float32(factor)


def test_axes_phases_refusals(L):
    for bad in (dict(sections=[]), dict(sections=[1] * 5), dict(sections=[0, 0]), dict(sections=[-1, 4]), dict(sections=[513]),
                dict(sections=[300, 300]), dict(sections=[4], base=0.0), dict(sections=[4], scaling="yarn", factor=2.0),
                dict(sections=[2, 2], ladder="per_axis", scaling="divisors", divisors=[1.0] * 4)):
        with pytest.raises(k.KvqError):
            k.kvq_rope_axes_phases(device="cpu", **bad)
    for bad in (dict(sections=[4], order="mixed"), dict(sections=[4], ladder="own"), dict(sections=[4], scaling="other"),
                dict(sections=[2, 2], scaling="divisors", divisors=[1.0]), dict(sections=[2 ** 32 + 4])):
        with pytest.raises(ValueError):
            k.kvq_rope_axes_phases(device="cpu", **bad)
    plan = k.kvq_rope_axes_phases([2, 2], scaling="divisors", divisors=[1.0, 2.0, 4.0, 8.0], device="cpu")
    assert plan.phases.numel() == 4
    # nothing is written on an error: the second axis has one frequency, for which the ntk scaling has no base
    ph, ax = (ctypes.c_uint64 * 4)(7, 7, 7, 7), (ctypes.c_uint8 * 4)(7, 7, 7, 7)
    z = k.kvq._RopeScaling(2, 2.0, 0.0, 1.0, 32.0, None)
    assert L.kvq_rope_axes_phases(2, (ctypes.c_int32 * 2)(3, 1), 0, 1, 1.0e4, ctypes.byref(z), ph, ax, None) == INVALID
    assert list(ph) == [7] * 4 and list(ax) == [7] * 4


def test_plan_checks():
    import torch
    for phases, axis_of in ((torch.zeros(4), [0] * 4), (torch.zeros(4, dtype=torch.int64), [0] * 5),
                            (torch.zeros(4, dtype=torch.int64), [0, 1, 2, 4])):
        with pytest.raises(ValueError):
            k.RopeAxes(phases, axis_of)


def test_host_tensors_are_refused(monkeypatch):
    """No host pointer reaches a kernel."""
    import torch
    monkeypatch.setattr(k.kvq, "_current_device", lambda: 0)
    plan = k.kvq_rope_axes_phases([64], device="cpu")
    x, pos = torch.zeros((2, 4, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        k.kvq_rope_axes_bf16(x, None, pos, plan, q_out=x)
    with pytest.raises(ValueError):
        k.kvq_rope_append_int8kv(k.KVCache(2, 4, 128, device="cpu"), None, x, x, pos, plan, pos, pos, pos.view(1, 2))


def test_a_workspace_on_another_device_is_refused(monkeypatch):
    import torch

    class Elsewhere:
        device = "cuda:7"
        get_device = staticmethod(lambda: 7)
        numel = staticmethod(lambda: 1 << 30)
        element_size = staticmethod(lambda: 1)

    monkeypatch.setattr(k.kvq, "_current_device", lambda: -1)  # what tensors of the host say
    cache = k.KVCache(4, 2, 128, device="cpu")
    q, row = torch.zeros((3, 4, 128), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace"):
        k.kvq_attn_prefill_window_int8kv(cache, q, 5, row, 0.1, 16, out=torch.empty_like(q), workspace=Elsewhere())
    with pytest.raises(ValueError, match="workspace"):
        k.kvq_decode_step_window_int8kv(cache, None, None, q, row.repeat(3, 1), torch.ones(3, dtype=torch.int32), 40, 0.1, 16,
                                        out=torch.empty((3, 4, 128)), workspace=Elsewhere())
