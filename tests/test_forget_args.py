"""Refusals and host arithmetic of the operators around a cache that forgets: no GPU, nothing is
launched (every call here is turned down by the checks that come before any CUDA call)."""
import ctypes

import numpy as np
import pytest

import forget_ref as R
import int8_kv_cache_quant_gb300 as k

A = 256  # an aligned address that is never used
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    return k.lib()


def cache(d=256, hkv=4, block=16, kp=A):
    return k.kvq._Cache(kp, A, A, A, 8, block, hkv, d)


def step(L, c=None, k_new=A, v_new=A, q=A, batch=1, n_new=1, hq=24, bt=A, mb=8, ctx=A, max_ctx=100, out=A, acc=A,
         stride=128, sp=A, pos=A, ws=A, wb=1 << 30, opts=None):
    return L.kvq_decode_step_accum_int8kv(ctypes.byref(c or cache()), k_new, v_new, q, batch, n_new, hq, bt, mb, ctx,
                                          max_ctx, 0.1, out, acc, stride, sp, pos, ws, wb,
                                          ctypes.byref(opts) if opts else None, None)


def opts(split=0, force=0):
    return k.kvq._decode_opts(split, 0, force)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(acc=None)), (INVALID, dict(stride=99)), (INVALID, dict(max_ctx=0)), (INVALID, dict(q=None)),
    (INVALID, dict(k_new=None)), (INVALID, dict(sp=None)), (INVALID, dict(pos=None)),
    (INVALID, dict(k_new=None, v_new=None)),  # positions without new tokens
    (INVALID, dict(hq=23)), (INVALID, dict(batch=0)), (INVALID, dict(opts=opts(split=24))),
    (INVALID, dict(opts=opts(force=3))), (UNSUPPORTED, dict(opts=opts(force=1))), (UNSUPPORTED, dict(hq=4 * 17)),
    (UNSUPPORTED, dict(n_new=9)), (UNSUPPORTED, dict(batch=65536)), (UNSUPPORTED, dict(c=cache(d=192))),
    (UNSUPPORTED, dict(max_ctx=(1 << 30) + 1, stride=1 << 31)),
    (UNSUPPORTED, dict(c=cache(block=32))), (MISALIGNED, dict(q=A + 2)), (MISALIGNED, dict(acc=A + 2)),
    (MISALIGNED, dict(ws=A + 8)), (MISALIGNED, dict(c=cache(kp=A + 4))), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(wb=1000, opts=opts(split=64)))])
def test_step_refusals(L, status, kw):
    assert step(L, **kw) == status


def test_step_workspace(L):
    # partials of 64-key splits at most (the smallest automatic split), then the scores of whole pages
    part = 16 * 24 * 256 * 4 + 16 * 24 * 16
    assert k.kvq_step_accum_workspace_bytes(1, 1, 24, 1000, 256) == part + 24 * 1008 * 4
    assert k.kvq_step_accum_workspace_bytes(1, 0, 24, 1000, 256) == 0
    # the size that is asked for is the size that is checked
    need = k.kvq_step_accum_workspace_bytes(2, 3, 8, 500, 128, split_rows=128)
    kw = dict(c=cache(d=128, hkv=2), batch=2, n_new=3, hq=8, max_ctx=500, stride=512, mb=32, opts=opts(split=128))
    assert step(L, wb=need - 1, **kw) == WORKSPACE


def weights(L, c=None, q=A, n=10, hq=24, hist=20, bt=A, nb=8, scale=0.1, acc=A, stride=64, ws=A, wb=1 << 30):
    return L.kvq_attn_chunk_weights_int8kv(ctypes.byref(c or cache()), q, n, hq, hist, bt, nb, scale, acc, stride, ws, wb, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(bt=None)), (INVALID, dict(acc=None)), (INVALID, dict(n=0)), (INVALID, dict(hq=0)),
    (INVALID, dict(hq=26)), (INVALID, dict(hist=-1)), (INVALID, dict(nb=0)), (INVALID, dict(nb=1)), (INVALID, dict(stride=29)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-0.1)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (UNSUPPORTED, dict(n=1 << 28, hist=0, nb=1 << 24, stride=1 << 28)), (UNSUPPORTED, dict(hist=(1 << 30) - 10, nb=1 << 27, stride=1 << 31)),
    (UNSUPPORTED, dict(n=1 << 22, hist=1 << 29, nb=1 << 26, stride=1 << 31)),  # a CTA's tiles are counted in 32 bits
    (UNSUPPORTED, dict(c=cache(hkv=65536), hq=65536)), (UNSUPPORTED, dict(c=cache(d=64))), (MISALIGNED, dict(q=A + 8)),
    (MISALIGNED, dict(acc=A + 1)), (MISALIGNED, dict(ws=A + 8)), (WORKSPACE, dict(ws=None))])
def test_chunk_weights_refusals(L, status, kw):
    assert weights(L, **kw) == status


def test_chunk_weights_workspace():
    # 10 queries x 6 heads: one row tile and one key tile per KV head, up to two runs of four parts
    # each; the row statistics; the queries in bf16
    rows = 4 * 128
    assert k.kvq_chunk_weights_workspace_bytes(10, 24, 4, 20, 256) == rows * 8 * 8 + 2 * rows * 4 + rows * 256 * 2 + rows * 8 * 4
    assert k.kvq_chunk_weights_workspace_bytes(0, 24, 4, 20, 256) == 0
    assert k.kvq_chunk_weights_workspace_bytes(10, 24, 4, -1, 256) == 0
    assert k.kvq_chunk_weights_workspace_bytes(10, 23, 4, 20, 256) == 0
    assert k.kvq_chunk_weights_workspace_bytes(10, 24, 4, 20, 192) == 0
    # no scores: the queries and the keys in bf16 and little else, where the scores would be 6.4 GB
    assert k.kvq_chunk_weights_workspace_bytes(2048, 24, 4, 30720, 256) < (2048 * 24 + 32768 * 4) * 256 * 2 + (16 << 20)


def evict(L, c=None, batch=2, bt=A, mb=8, ctx=A, max_ctx=100, keep=64, sink=0, recent=0, acc=A, sp=A + 1024, stride=128,
          ao=A + 2048, po=A + 4096, ostride=64, nl=A + 16, ws=A, wb=1 << 30):
    return L.kvq_cache_evict(ctypes.byref(c or cache()), batch, bt, mb, ctx, max_ctx, keep, sink, recent, acc, sp, stride,
                             ao, po, ostride, nl, ws, wb, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(acc=None)), (INVALID, dict(sp=None)), (INVALID, dict(ao=None)), (INVALID, dict(nl=None)),
    (INVALID, dict(ctx=None)), (INVALID, dict(bt=None)), (INVALID, dict(keep=0)), (INVALID, dict(max_ctx=0)),
    (INVALID, dict(batch=0)), (INVALID, dict(mb=0)), (INVALID, dict(sink=-1)), (INVALID, dict(recent=-1)),
    (INVALID, dict(sink=1, recent=64)), (INVALID, dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)),
    (INVALID, dict(stride=99)), (INVALID, dict(ostride=63)),
    (INVALID, dict(ao=A, ostride=128)),                             # acc in place, the positions not
    (INVALID, dict(ao=A, po=A + 1024, ostride=64)),                 # in place with other rows
    (INVALID, dict(nl=A)),                                          # the lengths in place
    (UNSUPPORTED, dict(batch=65536)), (UNSUPPORTED, dict(c=cache(hkv=65536))), (UNSUPPORTED, dict(c=cache(d=64))),
    (UNSUPPORTED, dict(max_ctx=(1 << 30) + 1, stride=1 << 31)),
    (MISALIGNED, dict(acc=A + 1)), (MISALIGNED, dict(nl=A + 2)), (MISALIGNED, dict(ws=A + 4)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(wb=15))])
def test_evict_refusals(L, status, kw):
    assert evict(L, **kw) == status


def test_evict_workspace(L):
    # 36 moves at most for 100 -> 64, then (on a 256-byte boundary) 64 slots, the counts
    units = 2 * 4
    r = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert k.kvq_evict_workspace_bytes(2, 4, 100, 64) == r(units * 36 * 4) + units * 64 * 4 + units * 4
    assert k.kvq_evict_workspace_bytes(2, 4, 64, 64) == units * 4  # nothing can move
    assert k.kvq_evict_workspace_bytes(2, 4, 100, 0) == 0
    need = k.kvq_evict_workspace_bytes(2, 4, 100, 64)
    assert evict(L, wb=need - 1) == WORKSPACE


def rope(L, q=A, qo=A, qs=24 * 256, qos=24 * 256, hq=24, kk=A, ko=A, ks=1024, kos=1024, hkv=4, d=256, n=2, pos=A, ph=A,
         r=64, off=0, layout=0):
    return L.kvq_rope_bf16(q, qo, qs, qos, hq, kk, ko, ks, kos, hkv, d, n, pos, ph, r, off, layout, 1.0, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(ko=None)), (INVALID, dict(pos=None)), (INVALID, dict(ph=None)),
    (INVALID, dict(n=-1)), (INVALID, dict(hq=-1)), (INVALID, dict(d=0)), (INVALID, dict(r=0)), (INVALID, dict(r=63)),
    (INVALID, dict(r=258)), (INVALID, dict(off=-2)), (INVALID, dict(off=194)), (INVALID, dict(off=2 ** 31 - 1)),
    (INVALID, dict(qs=24 * 256 - 1)), (INVALID, dict(kos=1000)), (INVALID, dict(qos=24 * 256 + 8)),
    (UNSUPPORTED, dict(layout=2)), (UNSUPPORTED, dict(d=1032, qs=1 << 20, qos=1 << 20, ks=1 << 20, kos=1 << 20)),
    (MISALIGNED, dict(q=A + 1)), (MISALIGNED, dict(pos=A + 2)), (MISALIGNED, dict(ph=A + 4))])
def test_rope_refusals(L, status, kw):
    assert rope(L, **kw) == status


def test_rope_nothing_to_do(L):
    assert rope(L, n=0) == 0
    assert rope(L, hq=0, hkv=0) == 0


SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
            ("yarn", dict(factor=16.0, original_len=4096.0)), ("yarn", dict(factor=1.0, original_len=512.0, low=2.0, high=8.0)),
            ("bands", dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0)), ("divisors", {})]


@pytest.mark.parametrize("r,base", [(128, 1.0e4), (64, 1.0e6), (6, 500.0)])
@pytest.mark.parametrize("kind,kw", SCALINGS)
def test_rope_phases(L, kind, kw, r, base):
    if kind == "divisors":
        kw = dict(divisors=list(np.linspace(1.0, 9.0, r // 2)))
    ph, af = k.kvq_rope_phases(r, base, kind, device="cpu", **kw)
    ref_kw = {("length" if n == "original_len" else n): v for n, v in kw.items()}
    inv, attn = R.inv_freq(r, base, kind, **ref_kw)
    turns = inv / (2 * np.pi)
    got = ph.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    # fp64 powers and quotients: a few steps of 2^-53 relative; and a phase is a whole number of 2^-64
    # turns, so it is half of that off whatever its size
    np.testing.assert_allclose(got, turns - np.floor(turns), rtol=16 * 2.0 ** -53, atol=2.0 ** -65)
    assert af == np.float32(attn)


def test_rope_phases_refusals(L):
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, base=float("nan")),
                dict(rotary_dim=2, scaling="ntk", factor=2.0), dict(rotary_dim=8, scaling="linear", factor=0.0),
                dict(rotary_dim=8, scaling="yarn", factor=2.0), dict(rotary_dim=8, scaling="bands", factor=2.0, low=4.0, high=1.0),
                dict(rotary_dim=8, scaling="divisors"), dict(rotary_dim=8, scaling="divisors", divisors=[1.0, 0.0, 1.0, 1.0])):
        with pytest.raises(k.KvqError):
            k.kvq_rope_phases(device="cpu", **bad)
    with pytest.raises(ValueError):
        k.kvq_rope_phases(8, scaling="other", device="cpu")
    with pytest.raises(ValueError):
        k.kvq_rope_phases(8, scaling="divisors", divisors=[1.0], device="cpu")


def test_wrap_checks_the_layout():
    import torch
    kk = torch.zeros((3, 2, 8, 16, 16), dtype=torch.int8)
    v = torch.zeros((3, 2, 128, 16), dtype=torch.int8)
    s = torch.zeros((3, 2, 16))
    c = k.KVCache.wrap(kk, v, s, s.clone())
    assert (c.num_blocks, c.n_kv_heads, c.head_dim) == (3, 2, 128) and c.k is kk
    for bad in ((kk, v[:, :, :64], s, s), (kk.float(), v, s, s), (kk, v, s[:2], s), (kk, v.transpose(2, 3), s, s)):
        with pytest.raises(ValueError):
            k.KVCache.wrap(*bad)
    with pytest.raises(ValueError):  # host memory never reaches a kernel
        c.struct()
