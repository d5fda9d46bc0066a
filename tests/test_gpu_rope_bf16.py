"""kvq_rope_bf16 against fp64 rotations: layouts, parts of a head, far and negative positions, packed
rows, in place, widths that are no whole number of 16 bytes."""
import numpy as np
import pytest

import forget_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    return k


def bf(rng, *shape):
    import torch
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(got, x, ang, factor, off, inter):
    """bf16 (8 significant bits) rounds the result by at most half a step, 2^-8 relative; before that fp32: cos and sin
    within 2^-24 + 2^-24 (polynomial, rounding) of themselves at most 1 in size, the angle's rounding
    (2^-24 of at most pi/4 off a quarter turn), the factor, one product and one fused sum: six half steps
    of 2^-24 on |x| + |y|, with the factor."""
    ref = R.rotate(x, ang, factor, off, inter)
    half = ang.shape[1]
    part = np.abs(x[..., off:off + 2 * half])
    size = np.zeros_like(x)
    if inter:
        size[..., off:off + 2 * half] = np.repeat(part[..., 0::2] + part[..., 1::2], 2, axis=-1)
    else:
        size[..., off:off + 2 * half] = np.tile(part[..., :half] + part[..., half:], 2)
    e32 = 6 * 2.0 ** -24 * abs(factor) * size
    tol = 2.0 ** -8 * np.abs(ref) + e32 * (1 + 2.0 ** -8)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - ref).max())
    rest = np.ones(x.shape[-1], bool)
    rest[off:off + 2 * half] = False
    assert np.array_equal(got[..., rest], x[..., rest])


CASES = [  # tokens, hq, hkv, d, r, off, inter
    (1, 24, 4, 256, 256, 0, False), (1, 1, 1, 128, 128, 0, True), (3, 8, 2, 128, 64, 0, False),
    (65, 5, 1, 256, 64, 192, True), (7, 2, 2, 80, 20, 40, False), (7, 2, 2, 80, 20, 40, True),
    (33, 3, 1, 96, 96, 0, True), (130, 4, 4, 64, 32, 16, False), (5, 3, 3, 10, 6, 3, False), (5, 3, 3, 10, 6, 3, True),
    (2, 1, 1, 2, 2, 0, True), (2, 1, 1, 3, 2, 1, False), (700, 24, 4, 256, 128, 64, False), (513, 32, 8, 128, 128, 0, True),
    (4, 2, 1, 1024, 1024, 0, False)]


@pytest.mark.parametrize("T,hq,hkv,d,r,off,inter", CASES)
def test_rotation(kvq, T, hq, hkv, d, r, off, inter):
    import torch
    rng = np.random.default_rng(T * 1000 + d)
    q, k = bf(rng, T, hq, d), bf(rng, T, hkv, d)
    pos = rng.integers(-2 ** 31, 2 ** 31, T).astype(np.int32)
    pos[:3] = [0, 2 ** 31 - 1, -2 ** 31][:min(T, 3)]
    ph, af = kvq.kvq_rope_phases(r, 1.0e4, "yarn", factor=8.0, original_len=4096.0)
    qo, ko = kvq.kvq_rope_bf16(q, k, torch.from_numpy(pos).cuda(), ph, layout=int(inter), rotary_offset=off, attn_factor=af)
    # the angle by exact integer arithmetic on the phases: p * phase mod 2^64
    phi = [int(x) & (2 ** 64 - 1) for x in ph.cpu().tolist()]
    ang = np.array([[(int(p) * f % 2 ** 64) / 2.0 ** 64 * 2 * np.pi for f in phi] for p in pos])
    check(f64(qo), f64(q), ang, af, off, inter)
    check(f64(ko), f64(k), ang, af, off, inter)


def test_against_the_frequencies(kvq):
    """Near positions, where fp64 angles are themselves exact to 1e-9: the plan and the kernel together."""
    import torch
    rng = np.random.default_rng(5)
    T, d = 257, 128
    q = bf(rng, T, 2, d)
    pos = np.arange(T, dtype=np.int32) * 511
    ph, af = kvq.kvq_rope_phases(d, 1.0e6)
    qo, none = kvq.kvq_rope_bf16(q, None, torch.from_numpy(pos).cuda(), ph)
    assert none is None
    check(f64(qo), f64(q), pos.astype(np.float64)[:, None] * R.inv_freq(d, 1.0e6)[0], 1.0, 0, False)


@pytest.mark.parametrize("inter", [False, True])
def test_packed_rows_and_in_place(kvq, inter):
    """q and k as views of one packed projection, rotated where they are; v and the rest untouched; rows
    that start off a 16-byte boundary give the same bits as contiguous ones."""
    import torch
    rng = np.random.default_rng(6)
    T, hq, hkv, d = 70, 6, 2, 128
    pos = torch.from_numpy(rng.integers(0, 100000, T).astype(np.int32)).cuda()
    ph, _ = kvq.kvq_rope_phases(d, 1.0e4)
    for shift in (0, 1, 2, 4):
        flat = bf(rng, T * (hq + 2 * hkv) * d + shift)
        qkv = flat[shift:].view(T, hq + 2 * hkv, d)
        before = qkv.clone()
        ref = kvq.kvq_rope_bf16(before[:, :hq].contiguous(), before[:, hq:hq + hkv].contiguous(), pos, ph, layout=int(inter))
        q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
        kvq.kvq_rope_bf16(q, k, pos, ph, layout=int(inter), q_out=q, k_out=k)
        assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
        assert torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:])


def test_gradient_is_the_rotation_back(kvq):
    """<rotate(x), g> as a function of x has gradient rotate(g, -pos): checked against fp64 differences
    (the function is linear, so a difference of any step is the derivative)."""
    import torch
    rng = np.random.default_rng(8)
    T, d = 9, 64
    x, g = bf(rng, T, 3, d), bf(rng, T, 3, d)
    pos = rng.integers(0, 50000, T).astype(np.int32)
    ph, _ = kvq.kvq_rope_phases(d, 1.0e4)
    grad, _ = kvq.kvq_rope_bf16(g, None, torch.from_numpy(-pos).cuda(), ph)
    ang = pos.astype(np.float64)[:, None] * R.inv_freq(d, 1.0e4)[0]
    check(f64(grad), f64(g), -ang, 1.0, 0, False)
    for _ in range(8):
        e = rng.standard_normal(x.shape)
        diff = ((R.rotate(f64(x) + e, ang, 1.0, 0, False) - R.rotate(f64(x), ang, 1.0, 0, False)) * f64(g)).sum()
        # every gradient element is 2^-8 (and fp32) off at most; 1.01 for taking it relative to the rounded one
        assert abs((f64(grad) * e).sum() - diff) <= (np.abs(f64(grad) * e)).sum() * 2.0 ** -8 * 1.01 + 1e-5


def test_infinities_stay_where_they_are(kvq):
    import torch
    x = torch.zeros((2, 1, 8), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0], x[0, 0, 7], x[1, 0, 3] = float("inf"), 3.0, float("nan")
    ph, _ = kvq.kvq_rope_phases(4, 1.0e4)
    y, _ = kvq.kvq_rope_bf16(x, None, torch.tensor([5, 5], dtype=torch.int32, device="cuda"), ph)
    y = y.float().cpu().numpy()
    assert not np.isfinite(y[0, 0, [0, 2]]).any() and np.isnan(y[1, 0, [1, 3]]).all()
    assert np.array_equal(y[0, 0, [1, 3, 4, 5, 6]], np.zeros(5)) and y[0, 0, 7] == 3.0
    assert np.array_equal(y[1, 0, [0, 2, 4, 5, 6, 7]], np.zeros(6))


def test_refused_tensors(kvq):
    import torch
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    ph, _ = kvq.kvq_rope_phases(64)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(pos=pos.long()), dict(pos=pos[:1]), dict(phases=ph.cpu()),
                dict(q=q.transpose(1, 2)), dict(k=q[:1]), dict(q_out=q[:, :1])):
        kw = dict(q=q, k=None, pos=pos, phases=ph) | bad
        with pytest.raises(ValueError):
            kvq.kvq_rope_bf16(**kw)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_rope_bf16(q, None, pos, ph, rotary_offset=2)
