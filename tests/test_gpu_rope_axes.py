"""kvq_rope_axes_bf16 against fp64 rotations: axes, orders, ladders, layouts, parts of a head, views of a packed
projection, far and negative positions; its inverse as the rotation's gradient; one axis as kvq_rope_bf16."""
import numpy as np
import pytest

import forget_ref as R
import window_ref as WR
from test_gpu_rope_bf16 import bf, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import int8_kv_cache_quant_gb300 as k
    k.lib()
    return k


def positions(rng, axes, T, far):
    import torch
    p = rng.integers(-far, far + 1, (axes, T)).astype(np.int32)
    return p, torch.from_numpy(p).cuda()


CASES = [  # tokens, hq, hkv, d, off, inter, sections, order, ladder, far
    (1, 24, 4, 256, 0, False, [44, 42, 42], "chunked", "shared", 40000),
    (3, 8, 2, 128, 0, True, [24, 20, 20], "turns", "shared", 1000),
    (65, 5, 1, 256, 192, True, [12, 20], "chunked", "per_axis", 100),
    (7, 2, 2, 80, 40, False, [4, 3, 3], "turns", "per_axis", 2 ** 31 - 1),
    (130, 4, 4, 64, 16, False, [4, 4, 4, 4], "turns", "shared", 10 ** 6),
    (33, 3, 1, 96, 0, True, [0, 24, 0, 24], "turns", "shared", 10 ** 6),
    (5, 3, 3, 10, 3, False, [1, 2], "chunked", "shared", 50),
    (2, 1, 1, 3, 1, True, [1], "chunked", "shared", 50),
    (700, 24, 4, 256, 64, False, [24, 20, 20], "turns", "shared", 10 ** 6),
    (513, 32, 8, 128, 0, True, [32, 32], "chunked", "per_axis", 70),
    (4, 2, 1, 1024, 0, False, [200, 156, 156], "chunked", "shared", 10 ** 5)]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,off,inter,sections,order,ladder,far", CASES)
def test_rotation(kvq, T, hq, hkv, d, off, inter, sections, order, ladder, far, inverse):
    rng = np.random.default_rng(T * 100 + d)
    q, k = bf(rng, T, hq, d), bf(rng, T, hkv, d)
    p, pos = positions(rng, len(sections), T, far)
    scaling = dict(scaling="yarn", factor=4.0, original_len=4096.0) if d == 256 else {}
    plan = kvq.kvq_rope_axes_phases(sections, base=1.0e5, order=order, ladder=ladder, **scaling)
    assert list(plan.axis_of) == WR.sections_to_axes(sections, order)
    layout = kvq.ROPE_INTERLEAVED if inter else kvq.ROPE_HALF
    qo, ko = kvq.kvq_rope_axes_bf16(q, k, pos, plan, layout=layout, rotary_offset=off, inverse=inverse)
    ang = WR.angles(p, plan.phases.cpu().numpy().view(np.uint64), plan.axis_of)
    for x, y in ((q, qo), (k, ko)):
        check(f64(y), f64(x), -ang if inverse else ang, plan.attn_factor, off, inter)


def test_one_axis_is_the_plain_rotation(kvq):
    import torch
    rng = np.random.default_rng(3)
    q, k = bf(rng, 40, 6, 128), bf(rng, 40, 2, 128)
    _, pos = positions(rng, 1, 40, 10 ** 6)
    phases, factor = kvq.kvq_rope_phases(96, 1.0e6, "linear", factor=2.0)
    plan = kvq.kvq_rope_axes_phases([48], base=1.0e6, scaling="linear", factor=2.0)
    assert torch.equal(plan.phases, phases) and plan.attn_factor == factor
    want = kvq.kvq_rope_bf16(q, k, pos[0], phases, rotary_offset=16, attn_factor=factor)
    got = kvq.kvq_rope_axes_bf16(q, k, pos[0], plan, rotary_offset=16)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # a text token has one number on all its axes
    three = kvq.kvq_rope_axes_phases([20, 14, 14], base=1.0e6, order="turns", scaling="linear", factor=2.0)
    got = kvq.kvq_rope_axes_bf16(q, k, pos.repeat(3, 1), three, rotary_offset=16)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_packed_rows_in_place_and_positions_apart(kvq):
    import torch
    rng = np.random.default_rng(4)
    T, hq, hkv, d = 77, 6, 2, 128
    qkv = bf(rng, T, hq + 2 * hkv, d)
    wide = torch.from_numpy(rng.integers(0, 5000, (3, 200)).astype(np.int32)).cuda()
    pos = wide[:, 60:60 + T]  # rows 200 apart
    plan = kvq.kvq_rope_axes_phases([24, 20, 20], order="turns")
    want = kvq.kvq_rope_axes_bf16(qkv[:, :hq].contiguous(), qkv[:, hq:hq + hkv].contiguous(), pos.contiguous(), plan)
    before = qkv.clone()
    kvq.kvq_rope_axes_bf16(qkv[:, :hq], qkv[:, hq:hq + hkv], pos, plan, q_out=qkv[:, :hq], k_out=qkv[:, hq:hq + hkv])
    assert torch.equal(qkv[:, :hq], want[0]) and torch.equal(qkv[:, hq:hq + hkv], want[1])
    assert torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:])  # v is not touched
    assert kvq.kvq_rope_axes_bf16(qkv[:0, :hq], None, pos[:, :0], plan)[0].shape == (0, hq, d)


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_is_the_gradient(kvq, inter):
    """Of L = sum(g . rotate(x)): by the formula (64 bits) and by differences of the operator's own outputs."""
    import torch
    rng = np.random.default_rng(5)
    T, H, d = 9, 3, 64
    x, g = bf(rng, T, H, d), bf(rng, T, H, d)
    p, pos = positions(rng, 2, T, 300)
    plan = kvq.kvq_rope_axes_phases([16, 16], scaling="yarn", factor=8.0, original_len=4096.0)
    layout = kvq.ROPE_INTERLEAVED if inter else kvq.ROPE_HALF
    dx = f64(kvq.kvq_rope_axes_bf16(g, None, pos, plan, layout=layout, inverse=True)[0])
    ang = WR.angles(p, plan.phases.cpu().numpy().view(np.uint64), plan.axis_of)
    check(dx, f64(g), -ang, plan.attn_factor, 0, inter)
    # the operator is linear, so a difference of any step gives the gradient but for bf16's rounding of the two
    # outputs (2^-8 of each, against g) and of dx (2^-8)
    for i in rng.choice(T * H * d, 40, replace=False):
        t, h, e = np.unravel_index(i, (T, H, d))
        up, down = x.clone(), x.clone()
        up[t, h, e], down[t, h, e] = 2.0, -2.0
        yu, yd = (f64(kvq.kvq_rope_axes_bf16(v, None, pos, plan, layout=layout)[0]) for v in (up, down))
        gd = f64(g)
        diff = ((yu - yd) * gd)[t, h].sum() / 4.0
        moved = (yu != yd)[t, h]
        tol = 2.0 ** -8 * ((np.abs(yu) + np.abs(yd)) * np.abs(gd))[t, h][moved].sum() / 4.0 + 2.0 ** -8 * abs(dx[t, h, e]) + 1e-5
        assert abs(diff - dx[t, h, e]) <= tol


def test_capture_replays(kvq):
    import torch
    rng = np.random.default_rng(6)
    q, k = bf(rng, 20, 4, 128), bf(rng, 20, 2, 128)
    _, pos = positions(rng, 3, 20, 1000)
    plan = kvq.kvq_rope_axes_phases([24, 20, 20])
    qo, ko = kvq.kvq_rope_axes_bf16(q, k, pos, plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_rope_axes_bf16(q, k, pos, plan, q_out=qo, k_out=ko)
    _, new = positions(rng, 3, 20, 1000)
    pos.copy_(new)
    graph.replay()
    want = kvq.kvq_rope_axes_bf16(q, k, new, plan)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
