"""Splits by the thousand: what the host decides before anything is launched, and, on the GPU, merges whose weights
pass the shared memory that a kernel has without asking."""
import ctypes
import threading

import numpy as np
import pytest

import int8_kv_cache_quant_gb300 as k

A = 256  # an aligned address that is never used


def test_a_step_whose_tail_cannot_be_counted_is_refused_before_anything_is_launched():
    c = k.kvq._Cache(A, A, A, A, 8, 16, 4, 128)
    o = k.kvq._decode_opts(65536, 0, 0)
    # 65535 x 4 KV heads x 2^20 CTAs of 1024 keys
    assert k.lib().kvq_decode_step_accum_int8kv(ctypes.byref(c), A, A, A, 65535, 1, 4, A, 1 << 26, A, 1 << 30, 0.1, A, A, 1 << 30,
                                                A, A, A, 1 << 62, ctypes.byref(o), None) == 2


def _side(kvq, slots, n):
    import torch
    from test_gpu_evict import dev
    rng = np.random.default_rng(slots)
    cache = kvq.KVCache(4, 1, 128)
    q, k_new, v_new = (torch.from_numpy(rng.standard_normal((1, h, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
                       for h in (1, 1, 1))
    table = torch.zeros((1, slots // 16), dtype=torch.int32, device="cuda")
    acc = torch.zeros((1, 1, slots), device="cuda")
    ws = torch.empty(kvq.kvq_step_accum_workspace_bytes(1, 1, 1, slots, 128, split_rows=16), dtype=torch.uint8, device="cuda")
    out, ctx, s = torch.zeros((1, 1, 128), device="cuda"), dev(np.array([n], np.int32)), torch.cuda.Stream()
    torch.cuda.synchronize()

    def call():
        kvq.kvq_decode_step_accum_int8kv(cache, k_new, v_new, q, table, ctx, slots, 0.1, acc, out=out, workspace=ws, split_rows=16,
                                         stream=s)

    return call, acc


@pytest.mark.gpu
def test_steps_of_many_splits_from_two_host_threads():
    """Each thread's call has its own number of splits, both past what a kernel has without asking."""
    import torch
    k.lib()
    k.kvq_device_status()
    sides = [_side(k, 16 * 10300, 9), _side(k, 16 * 16384, 9)]
    errors = []

    def run(call):
        try:
            torch.cuda.set_device(0)
            for _ in range(1500):
                call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c, _ in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    assert k.kvq_device_status() == 0
    for _, acc in sides:
        a = acc.cpu().numpy().astype(np.float64)[0, 0]
        assert (a[9:] == 0).all() and (a[:8] == a[0]).all()
        # Eight old keys of zeros share a call's weight 1 equally with the new one, which starts from zero each time: in
        # 1500 calls 8 a[0] + 1500 a[8] = 1500.  1500 additions are each within half a step of a sum below 256 (2^-17),
        # and a weight's relative error is that of its score (below 8 in log2 units) and a few exponentials: 1e-5
        assert abs(8 * a[0] + 1500 * a[8] - 1500) < 8 * 1500 * 2.0 ** -17 + 1500 * 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_split", [10240, 10241, 11200, 11800, 12288, 12289, 16384])
def test_a_decode_step_of_many_splits(n_split, d):
    """Whatever the bound of the lengths: the result of the call with the smallest bound, to the bit (a short context's
    splits are the same)."""
    import torch
    rng = np.random.default_rng(n_split)
    n, hkv, G = 100, 1, 4
    bits = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    q, k_new, v_new, kf, vf = bits(1, G, d), bits(1, hkv, d), bits(1, hkv, d), bits(n - 1, hkv, d), bits(n - 1, hkv, d)
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    res = []
    for slots in (112, 16 * n_split):
        cache = k.KVCache(7, hkv, d)
        table = torch.full((1, slots // 16), -1, dtype=torch.int32, device="cuda")
        table[0, :7] = torch.arange(7)
        k.kvq_quant_write(cache, kf, vf, torch.zeros(n - 1, dtype=torch.int32, device="cuda"),
                          torch.arange(n - 1, dtype=torch.int32, device="cuda"), table)
        out = k.kvq_decode_step_int8kv(cache, k_new, v_new, q, table, ctx, slots, 0.1, split_rows=16, force_route=2)
        res.append((out, k.kvq_attn_decode_int8kv(cache, q, table, ctx, slots, 0.1, split_rows=16, force_route=2), cache.k, cache.v))
    assert k.kvq_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*res))
