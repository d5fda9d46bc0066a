"""Measured cases of windowed attention over the paged int8 cache and of what feeds it: the decode step and the
prompt chunk with a sliding window and first tokens that stay visible, rotary positions with several axes, and the
rotation, quantisation and append of new tokens in one call.

Each operator has its plain form here (elementary torch operations in fp32, angles in fp64) and, with `own` set, the
library's call.  Shapes follow the repository's workloads: 24 query / 4 KV heads at head_dim 256 (one sequence of
32768 keys) and 32 / 8 heads at head_dim 128 (64 sequences of 512 to 16384 keys), pages of 16 tokens dealt in random
order.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest step of a windowed layer: one new token far into a sequence, where latency counts
        dict(name="step_window_1k", op="step", batch=1, hq=24, hkv=4, d=256, lo=32768, hi=32768, new=1, window=1024, sink=4),
        # a serving batch of ragged lengths, some shorter than the window
        dict(name="step_window_b64", op="step", batch=64, hq=32, hkv=8, d=128, lo=512, hi=16384, new=1, window=4096, sink=4),
        # a verify step of four drafted tokens, an odd window and sinks that end inside a page
        dict(name="step_window_verify", op="step", batch=1, hq=24, hkv=4, d=256, lo=32767, hi=32767, new=4, window=8191, sink=100),
        # a short follow-up question behind a history longer than the window
        dict(name="prompt_window_33", op="prompt", tokens=33, history=5000, hq=24, hkv=4, d=256, window=1023, sink=4),
        # a whole prompt of odd length behind an odd, short history, no sinks
        dict(name="prompt_window_2k", op="prompt", tokens=2047, history=333, hq=32, hkv=8, d=128, window=1024, sink=0),
        # a chunk of a long prompt
        dict(name="prompt_window_32k", op="prompt", tokens=2048, history=30720, hq=24, hkv=4, d=256, window=4096, sink=4),
        # one token's heads, three axes
        dict(name="axes_1", op="axes", tokens=1, hq=24, hkv=4, d=256, rot=256, off=0, inter=False, axes=3, order="chunked",
             ladder="shared", inverse=False, far=32768),
        # an image's patches, two axes with frequencies of their own: the gradient's direction
        dict(name="axes_image_4k", op="axes", tokens=4095, hq=32, hkv=8, d=128, rot=128, off=0, inter=False, axes=2,
             order="chunked", ladder="own", inverse=True, far=1),
        # a prompt chunk with video far into a conversation, axes taking turns, a part of each head rotated
        dict(name="axes_chunk_2k", op="axes", tokens=2048, hq=24, hkv=4, d=256, rot=128, off=0, inter=True, axes=3,
             order="turns", ladder="shared", inverse=False, far=1000000),
        # one new token
        dict(name="append_1", op="append", batch=1, tokens=1, hq=24, hkv=4, d=256, rot=256, off=0, inter=False, axes=1,
             order="chunked", ladder="shared", at=1000, far=32768),
        # a serving batch's new tokens, one a sequence
        dict(name="append_b64", op="append", batch=64, tokens=1, hq=32, hkv=8, d=128, rot=128, off=0, inter=False, axes=3,
             order="chunked", ladder="shared", at=1500, far=131072),
        # a prompt chunk with images, from the middle of a page on
        dict(name="append_chunk_2k", op="append", batch=1, tokens=2048, hq=24, hkv=4, d=256, rot=128, off=0, inter=False,
             axes=3, order="turns", ladder="shared", at=333, far=1000000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "prompt", "axes", "append"])
    hkv, g, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([128, 256])
    window, sink = _log(rng, 16, 8192), rng.choice([0, 1, 4, 4, 16, 100, 200])
    if op == "step":
        hi = _log(rng, 64, 32768)
        batch = max(1, min(_log(rng, 1, 64), (1 << 19) // hi))
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d if batch * hi * hkv < (1 << 21) else 128,
                    lo=max(8, int(hi * rng.uniform(0.05, 1.0))), hi=hi, new=rng.choice([1, 1, 1, 2, 3, 5]),
                    window=min(window, 4096) if batch > 8 else window, sink=sink)
    if op == "prompt":
        return dict(op=op, tokens=_log(rng, 1, 2048), history=_log(rng, 1, 30720) - 1, hq=min(24, hkv * g) // hkv * hkv,
                    hkv=hkv, d=d, window=min(window, 4096), sink=sink)
    off = rng.choice([0, 0, 0, d // 2])
    rot = (d - off) // rng.choice([1, 1, 2])
    more = dict(hq=hkv * min(g, 4), hkv=hkv, d=d, rot=rot, off=off, inter=rng.random() < 0.5, axes=rng.choice([1, 2, 3, 3, 4]),
                order=rng.choice(["chunked", "turns"]), ladder=rng.choice(["shared", "own"]), far=_log(rng, 1, 4000000))
    if op == "axes":
        return dict(op=op, tokens=_log(rng, 1, 4000), inverse=rng.random() < 0.5, **more)
    batch = rng.choice([1, 1, _log(rng, 2, 64)])
    return dict(op=op, batch=batch, tokens=_log(rng, 1, 2048 if batch == 1 else 8), at=_log(rng, 1, 2000) - 1, **more)


# ------------------------------------------------------------------------------------ inputs
def _lens(case):
    """The lengths of a batch: spread evenly over [lo, hi] (the case fixes them, the seed their order)."""
    n = case["batch"]
    if n == 1:
        return [case["hi"]]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // (n - 1) for i in range(n)]


def _quantise(x):
    """Rows (last dim) to int8 codes and one fp32 scale: amax / 127, rint(x / scale)."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = amax / torch.full_like(amax, 127.0)
    code = torch.where(scale > 0, x / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(x))
    return code.round().clamp(-127, 127).to(torch.int8), scale[..., 0]


def _cache(gen, num_blocks, hkv, d):
    """A pool of pages filled with the codes of normal rows, one key element in a hundred eight times as large."""
    dev = "cuda"
    k = torch.empty((num_blocks, hkv, d // 16, PAGE, 16), dtype=torch.int8, device=dev)
    v = torch.empty((num_blocks, hkv, d, PAGE), dtype=torch.int8, device=dev)
    ks = torch.empty((num_blocks, hkv, PAGE), dtype=torch.float32, device=dev)
    vs = torch.empty_like(ks)
    step = max(1, (1 << 27) // (hkv * d * PAGE))
    for s in range(0, num_blocks, step):
        n = min(step, num_blocks - s)
        x = torch.randn((n, hkv, PAGE, d), generator=gen, device=dev)
        x = torch.where(torch.rand(x.shape, generator=gen, device=dev) < 0.01, 8 * x, x)
        c, ks[s:s + n] = _quantise(x)
        k[s:s + n] = c.view(n, hkv, PAGE, d // 16, 16).permute(0, 1, 3, 2, 4)
        c, vs[s:s + n] = _quantise(torch.randn((n, hkv, PAGE, d), generator=gen, device=dev))
        v[s:s + n] = c.permute(0, 1, 3, 2)
    return dict(k=k, v=v, ks=ks, vs=vs)


def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _table(gen, lens):
    """Pages of one pool dealt in random order; the rest of a row is -1."""
    pages = [-(-n // PAGE) for n in lens]
    pool = torch.randperm(sum(pages), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, sum(pages)


def _sections(case):
    """Frequencies of each axis: the first (time) takes what an even split leaves."""
    half, n = case["rot"] // 2, case["axes"]
    rest = half // n
    return [half - rest * (n - 1)] + [rest] * (n - 1)


def _axis_of(case):
    """The axis of each frequency: one axis after the other, or axes taking turns until theirs are used up."""
    sec = _sections(case)
    if case["order"] == "chunked":
        return [a for a, n in enumerate(sec) for _ in range(n)]
    left, out = list(sec), []
    while len(out) < sum(sec):
        for a in range(len(sec)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _ladder(case):
    """(place, length) of each frequency in its ladder base^(-place / length): the head's, or its axis's own."""
    axis_of, sec, seen, out = _axis_of(case), _sections(case), [0] * case["axes"], []
    for j, a in enumerate(axis_of):
        out.append((j, len(axis_of)) if case["ladder"] == "shared" else (seen[a], sec[a]))
        seen[a] += 1
    return out


BASE = 1.0e6


def _positions(gen, case, n):
    """Positions [axes][n]: text (all axes alike), then frames of a grid of patches."""
    start = int(torch.randint(0, case["far"], (1,), generator=gen, device="cuda"))
    i = torch.arange(n, device="cuda")
    text = n // 4
    img = (i - text).clamp(min=0)
    wide = max(1, math.isqrt(max(1, n - text)) // 2)
    tall = max(1, wide // 2)
    grid = [img // (wide * tall), img // wide % tall, img % wide, img % 7]
    return torch.stack([torch.where(i < text, start + i, start + text + grid[a]) for a in range(case["axes"])]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    op, s = case["op"], dict(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "step":
        lens = _lens(case)
        order = torch.randperm(len(lens), generator=gen, device="cuda").tolist()
        lens = [lens[i] for i in order]
        s["table"], blocks = _table(gen, lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["max_ctx"] = max(lens)
        s |= _cache(gen, blocks, hkv, d)
        b, n = case["batch"], case["new"]
        s["q"], s["k_new"], s["v_new"] = _bf16(gen, b, n, hq, d), _bf16(gen, b, n, hkv, d), _bf16(gen, b, n, hkv, d)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty((b, n, hq, d), dtype=torch.float32, device="cuda")
    elif op == "prompt":
        n = case["tokens"]
        s["table"], blocks = _table(gen, [case["history"] + n])
        s |= _cache(gen, blocks, hkv, d)
        s["q"], s["scale"] = _bf16(gen, n, hq, d), 1.0 / math.sqrt(d)
        s["out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    else:
        b = case.get("batch", 1)
        n = b * case["tokens"]
        # the projection's output, q | k | v of a token side by side
        qkv = _bf16(gen, n, hq + 2 * hkv, d)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["pos"] = _positions(gen, case, n)
        # the plan: each frequency in turns per position as a 64-bit fraction, and its axis
        place = np.array(_ladder(case), np.float64)
        turns = (BASE ** (-place[:, 0] / place[:, 1]) / (2 * math.pi) * 2.0 ** 64).round().astype(np.uint64)
        s["phases"] = torch.from_numpy(turns.view(np.int64)).cuda()
        s["axis_of"] = _axis_of(case)
        s["axis"] = torch.tensor(s["axis_of"], device="cuda")
        s["factor"] = 1.0
        s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty((n, hkv, d), dtype=torch.bfloat16, device="cuda")
    if op == "append":
        t = case["tokens"]
        # sequences of odd lengths whose newest tokens are these; slots are not positions
        first = [case["at"] + 37 * i % 61 for i in range(b)]
        s["table"], blocks = _table(gen, [f + t for f in first])
        s |= dict(k=torch.randint(-127, 128, (blocks, hkv, d // 16, PAGE, 16), generator=gen, device="cuda", dtype=torch.int8),
                  v=torch.randint(-127, 128, (blocks, hkv, d, PAGE), generator=gen, device="cuda", dtype=torch.int8),
                  ks=torch.rand((blocks, hkv, PAGE), generator=gen, device="cuda"),
                  vs=torch.rand((blocks, hkv, PAGE), generator=gen, device="cuda"))
        s["seq"] = torch.arange(b, dtype=torch.int32, device="cuda").repeat_interleave(t)
        s["slot"] = (torch.tensor(first, device="cuda")[:, None] + torch.arange(t, device="cuda")).flatten().to(torch.int32)
    return s


# ------------------------------------------------------------------------------------ one pass
def _rows(s, page, at):
    """K and V of the keys at (page, slot of it), dequantised: [...][Hkv][D]."""
    k = s["k"][page, :, :, at].float() * s["ks"][page, :, at][..., None, None]
    v = s["v"][page, :, :, at].float() * s["vs"][page, :, at][..., None]
    return k.flatten(-2), v


def _seen(t, p, window, sink):
    """Key t as the row at position p sees it."""
    return (t >= 0) & (t <= p) & ((t > p - window) | (t < sink))


def _softmax(sc, seen):
    sc = sc.masked_fill(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = (sc - torch.where(m > -math.inf, m, torch.zeros_like(m))).exp()
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, torch.ones_like(l))


def _plain_step(s):
    b, n, hq, hkv, d, w, sink = (s[x] for x in ("batch", "new", "hq", "hkv", "d", "window", "sink"))
    g, dev = hq // hkv, "cuda"
    pos = s["lens"].long()[:, None] - n + torch.arange(n, device=dev)
    # the new tokens' rows into their slots
    page, at = s["table"].long().gather(1, pos // PAGE), pos % PAGE
    kc, kscale = _quantise(s["k_new"].float())
    vc, vscale = _quantise(s["v_new"].float())
    s["k"][page, :, :, at] = kc.view(b, n, hkv, d // 16, 16)
    s["v"][page, :, :, at] = vc
    s["ks"][page, :, at], s["vs"][page, :, at] = kscale, vscale
    # the first tokens, then the keys of the rows' windows
    low = (pos[:, :1] - w + 1).clamp(min=sink)
    t = torch.cat((torch.arange(sink, device=dev).expand(b, sink), low + torch.arange(min(w, s["max_ctx"]) + n - 1, device=dev)), 1)
    live = t < s["lens"][:, None]
    t = torch.where(live, t, torch.zeros_like(t))
    k, v = _rows(s, s["table"].long().gather(1, t // PAGE), t % PAGE)
    q = s["q"].float().view(b, n, hkv, g, d).transpose(1, 2).reshape(b, hkv, n * g, d)
    sc = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    seen = _seen(t[:, None], pos[:, :, None], w, sink) & live[:, None]
    p = _softmax(sc, seen.repeat_interleave(g, 1)[:, None])
    s["out"].copy_((p @ v.transpose(1, 2)).view(b, hkv, n, g, d).transpose(1, 2).reshape(b, n, hq, d))
    return [s["out"], s["k"], s["v"], s["ks"], s["vs"]]


def _plain_prompt(s):
    n, hist, hq, hkv, d, w, sink = (s[x] for x in ("tokens", "history", "hq", "hkv", "d", "window", "sink"))
    g, dev = hq // hkv, "cuda"
    low = max(0, hist - w + 1)
    t = torch.cat((torch.arange(min(sink, low), device=dev), torch.arange(low, hist + n, device=dev)))
    k, v = _rows(s, s["table"][0].long()[t // PAGE], t % PAGE)
    q = s["q"].float().view(n, hkv, g, d).transpose(0, 1).reshape(hkv, n * g, d)
    sc = (q @ k.permute(1, 2, 0)).mul_(s["scale"])
    p = _softmax(sc, _seen(t, hist + torch.arange(n, device=dev).repeat_interleave(g)[:, None], w, sink))
    s["out"].copy_((p @ v.transpose(0, 1)).view(hkv, n, g, d).transpose(0, 1).reshape(n, hq, d))
    return [s["out"]]


def _cos_sin(s, inverse=False):
    """fp32 cos and sin of each token's frequencies [n][1][r / 2]: the product with the position is exact in 64 bits."""
    turns = s["pos"].long()[s["axis"]].T * s["phases"]
    ang = turns.double() * (2.0 * math.pi / 2.0 ** 64)
    c, sn = (ang.cos() * s["factor"]).float(), (ang.sin() * s["factor"]).float()
    return c[:, None], (-sn if inverse else sn)[:, None]


def _rotate(s, x, c, sn):
    r, off = s["rot"], s["off"]
    x = x.float()
    part = x[..., off:off + r]
    a, b = (part[..., 0::2], part[..., 1::2]) if s["inter"] else (part[..., :r // 2], part[..., r // 2:])
    lo, hi = a * c - b * sn, b * c + a * sn
    z = torch.stack((lo, hi), -1).flatten(-2) if s["inter"] else torch.cat((lo, hi), -1)
    return torch.cat((x[..., :off], z, x[..., off + r:]), -1)


def _plain_axes(s):
    c, sn = _cos_sin(s, s["inverse"])
    s["q_out"].copy_(_rotate(s, s["q"], c, sn))
    s["k_out"].copy_(_rotate(s, s["k_new"], c, sn))
    return [s["q_out"], s["k_out"]]


def _plain_append(s):
    c, sn = _cos_sin(s)
    s["q_out"].copy_(_rotate(s, s["q"], c, sn))
    slot = s["slot"].long()
    page, at = s["table"].long()[s["seq"].long(), slot // PAGE], slot % PAGE
    kc, kscale = _quantise(_rotate(s, s["k_new"], c, sn))
    vc, vscale = _quantise(s["v_new"].float())
    s["k"][page, :, :, at] = kc.view(-1, s["hkv"], s["d"] // 16, 16)
    s["v"][page, :, :, at] = vc
    s["ks"][page, :, at], s["vs"][page, :, at] = kscale, vscale
    return [s["q_out"], s["k"], s["v"], s["ks"], s["vs"]]


def _own(s):
    import int8_kv_cache_quant_gb300 as kvq
    op = s["op"]
    if op in ("axes", "append") and "plan" not in s:  # the handle that a program keeps
        s["plan"] = kvq.RopeAxes(s["phases"], s["axis_of"], s["factor"])
        s["layout"] = kvq.ROPE_INTERLEAVED if s["inter"] else kvq.ROPE_HALF
    if op == "axes":
        kvq.kvq_rope_axes_bf16(s["q"], s["k_new"], s["pos"], s["plan"], layout=s["layout"], rotary_offset=s["off"],
                               inverse=s["inverse"], q_out=s["q_out"], k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    if "cache" not in s:  # the handle and the workspace that a program keeps
        s["cache"] = kvq.KVCache.wrap(s["k"], s["v"], s["ks"], s["vs"])
        need = 0
        if op == "step":
            need = kvq.kvq_step_window_workspace_bytes(s["batch"], s["new"], s["hq"], s["hkv"], s["max_ctx"], s["window"],
                                                       s["sink"], s["d"])
        elif op == "prompt":
            need = kvq.kvq_prefill_window_workspace_bytes(s["tokens"], s["hq"], s["hkv"], s["history"], s["window"], s["sink"],
                                                          s["d"])
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    if op == "append":
        kvq.kvq_rope_append_int8kv(s["cache"], s["q"], s["k_new"], s["v_new"], s["pos"], s["plan"], s["seq"], s["slot"],
                                   s["table"], layout=s["layout"], rotary_offset=s["off"], q_out=s["q_out"])
        return [s["q_out"], s["k"], s["v"], s["ks"], s["vs"]]
    if op == "prompt":
        kvq.kvq_attn_prefill_window_int8kv(s["cache"], s["q"], s["history"], s["table"][0], s["scale"], s["window"], s["sink"],
                                           out=s["out"], workspace=s["ws"])
        return [s["out"]]
    kvq.kvq_decode_step_window_int8kv(s["cache"], s["k_new"], s["v_new"], s["q"], s["table"], s["lens"], s["max_ctx"],
                                      s["scale"], s["window"], s["sink"], out=s["out"], workspace=s["ws"])
    return [s["out"], s["k"], s["v"], s["ks"], s["vs"]]


def run(s):
    if own:
        return _own(s)
    return {"step": _plain_step, "prompt": _plain_prompt, "axes": _plain_axes, "append": _plain_append}[s["op"]](s)


# ------------------------------------------------------------------------------------ what a pass needs
def _visible(p, window, sink):
    """Keys that the row at position p sees."""
    return p + 1 if p + 1 <= window + sink else window + min(sink, p + 1 - window)


def work(case):
    op, d, hq, hkv = case["op"], case["d"], case["hq"], case["hkv"]
    if op == "step":
        n, w, sink = case["new"], case["window"], case["sink"]
        keys = sum(_visible(c - 1, w + n - 1, sink) for c in _lens(case))
        pairs = sum(_visible(c - n + i, w, sink) for c in _lens(case) for i in range(n))
        # K, V and both scales of every key that a row sees once, the new rows, q and the output
        return dict(bytes=keys * hkv * (2 * d + 8) + case["batch"] * n * (hq * d * 6 + hkv * (6 * d + 8)) + keys / 4,
                    flops=4.0 * pairs * hq * d)
    if op == "prompt":
        n, hist, w, sink = case["tokens"], case["history"], case["window"], case["sink"]
        pairs = sum(_visible(hist + i, w, sink) for i in range(n))
        return dict(bytes=_visible(hist + n - 1, w + n - 1, sink) * hkv * (2 * d + 8) + n * hq * d * 4.0,
                    flops=4.0 * pairs * hq * d)
    n = case.get("batch", 1) * case["tokens"]
    if op == "axes":
        return dict(bytes=n * (hq + hkv) * d * 4 + n * 4 * case["axes"], flops=3.0 * n * (hq + hkv) * case["rot"])
    # q, k and v in, q out, codes and scales out
    return dict(bytes=n * (hq * d * 4 + hkv * (6 * d + 8)) + n * 4 * (case["axes"] + 2), flops=3.0 * n * (hq + hkv) * case["rot"])


# ------------------------------------------------------------------------------------ by the definition, in 64 bits
def _turned(case, s, x, sign):
    """Rows x rotated as complex numbers, 64 bits, from the frequencies themselves."""
    axis, pos = _axis_of(case), s["pos"].cpu().numpy().astype(np.float64)
    inv = np.array([math.exp(-i / n * math.log(BASE)) for i, n in _ladder(case)])
    z = torch.from_numpy(np.exp(1j * sign * pos[axis].T * inv)).cuda()[:, None]
    y, i = x.double().clone(), torch.arange(case["rot"] // 2, device="cuda")
    off = case["off"]
    ia, ib = (off + 2 * i, off + 2 * i + 1) if case["inter"] else (off + i, off + i + case["rot"] // 2)
    w = torch.complex(y[..., ia], y[..., ib]) * z
    y[..., ia], y[..., ib] = w.real, w.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "axes":
        sign = -1.0 if case["inverse"] else 1.0
        return [_turned(case, s, s["q"], sign), _turned(case, s, s["k_new"], sign)]
    ks, vs = s["ks"].double(), s["vs"].double()
    if op == "append":
        for h in range(case["hkv"]):
            for scales, rows in ((ks, _turned(case, s, s["k_new"], 1.0)), (vs, s["v_new"].double())):
                slot = s["slot"].long()
                scales[s["table"][s["seq"].long(), slot // PAGE].long(), h, slot % PAGE] = rows[:, h].abs().amax(-1) / 127.0
        return [_turned(case, s, s["q"], 1.0), None, None, ks, vs]
    hq, hkv, d, w, sink = (case[x] for x in ("hq", "hkv", "d", "window", "sink"))
    g = hq // hkv
    if op == "prompt":
        n, hist = case["tokens"], case["history"]
        out = torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
        where = s["table"][0].long().repeat_interleave(PAGE)
        for i0 in range(0, n, 512):  # queries in blocks, each over the keys between its first window and itself
            i = torch.arange(i0, min(n, i0 + 512), device="cuda")
            first = max(0, hist + i0 - w + 1)
            t = torch.arange(hist + int(i[-1]) + 1, device="cuda")
            t = t[(t < sink) | (t >= first)]
            far = (hist + i)[:, None] - t[None]  # how far back
            hidden = (far < 0) | ((far >= w) & (t >= sink))
            for h in range(hkv):
                k = s["k"][where[t], h, :, t % PAGE].reshape(-1, d).double() * s["ks"][where[t], h, t % PAGE].double()[:, None]
                v = s["v"][where[t], h, :, t % PAGE].double() * s["vs"][where[t], h, t % PAGE].double()[:, None]
                for j in range(h * g, h * g + g):
                    z = s["q"][i, j].double() @ k.T / math.sqrt(d)
                    out[i, j] = torch.softmax(z.masked_fill_(hidden, -math.inf), 1) @ v
        return [out]
    b, n = case["batch"], case["new"]
    out = torch.zeros((b, n, hq, d), dtype=torch.float64, device="cuda")
    for i in range(b):
        ctx = int(s["lens"][i])
        t = torch.arange(ctx, device="cuda")
        t = t[(t < sink) | (t > ctx - n - w)]
        page, at = s["table"][i].long()[t // PAGE], t % PAGE
        k = s["k"][page, :, :, at].reshape(-1, hkv, d).double() * s["ks"][page, :, at].double()[..., None]
        v = s["v"][page, :, :, at].double() * s["vs"][page, :, at].double()[..., None]
        for rows, new, scales in ((k, s["k_new"][i], ks), (v, s["v_new"][i], vs)):
            x = new.double()
            # the codes are defined by fp32 quotients: a tie of those goes to the even code
            unit = (x.abs().amax(-1, keepdim=True).float() / torch.full((1,), 127.0, device="cuda")).double()
            rows[-n:] = (x / unit).float().round().double() * unit
            scales[page[-n:], :, at[-n:]] = x.abs().amax(-1) / 127.0
        for j in range(n):
            p = ctx - n + j
            m = (t <= p) & ((p - t < w) | (t < sink))
            z = torch.einsum("hgd,thd->hgt", s["q"][i, j].double().view(hkv, g, d), k[m]) / math.sqrt(d)
            out[i, j] = torch.einsum("hgt,thd->hgd", torch.softmax(z, 2), v[m]).reshape(hq, d)
    return [out, None, None, ks, vs]
