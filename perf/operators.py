"""Measured cases of the operators around a cache that forgets: decode with accumulated attention
weights, the attention weights of a chunk of prompt queries, eviction from the paged int8 cache by
accumulated weight, and rotary positions that are independent of the cache slot.

Each operator has its plain form here (elementary torch operations in fp32, angles in fp64) and, with
`own` set, the library's call.  Shapes follow the repository's workloads: 24 query / 4 KV heads at
head_dim 256 (one sequence of 32768 keys) and 32 / 8 heads at head_dim 128 (64 sequences of 512 to
16384 keys), pages of 16 tokens dealt in random order.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest decode step: one short sequence, where launches and latency count
        dict(name="step_1k", op="step", batch=1, hq=24, hkv=4, d=256, lo=1024, hi=1024, new=1),
        # a serving batch of ragged lengths, one new token each
        dict(name="step_b64", op="step", batch=64, hq=32, hkv=8, d=128, lo=512, hi=16384, new=1),
        # a verify step of four drafted tokens behind a long context
        dict(name="step_verify_32k", op="step", batch=1, hq=24, hkv=4, d=256, lo=32767, hi=32767, new=4),
        # an observation window: the prompt's last queries decide what a long prompt keeps
        dict(name="weights_window_32k", op="weights", tokens=32, history=32736, hq=24, hkv=4, d=256),
        # a whole prompt of odd length behind an odd, short history
        dict(name="weights_prompt_2k", op="weights", tokens=2047, history=333, hq=32, hkv=8, d=128),
        # a full chunk of a long prompt: every query's weights over 32768 keys
        dict(name="weights_chunk_32k", op="weights", tokens=2048, history=30720, hq=24, hkv=4, d=256),
        # steady state of a serving batch: one token over the budget in every sequence
        dict(name="evict_step_b8", op="evict", batch=8, hkv=8, d=128, lo=1025, hi=1025, keep=1024, sink=4, recent=64),
        # a batch of ragged prompts brought down to one budget (the short ones keep everything)
        dict(name="evict_b64", op="evict", batch=64, hkv=8, d=128, lo=512, hi=16384, keep=2048, sink=4, recent=256),
        # one long prompt brought down to an eighth
        dict(name="evict_prompt_32k", op="evict", batch=1, hkv=4, d=256, lo=32768, hi=32768, keep=4096, sink=4, recent=512),
        # the rotation of one token's heads
        dict(name="rope_1", op="rope", tokens=1, hq=24, hkv=4, d=256, rot=256, off=0, inter=False, scaling="none",
             far=32768),
        # a serving batch's new tokens, adjacent pairs, context extended eightfold
        dict(name="rope_b64", op="rope", tokens=64, hq=32, hkv=8, d=128, rot=128, off=0, inter=True, scaling="yarn",
             far=131072),
        # a prompt chunk at far positions, a quarter of each head rotated, positions interpolated
        dict(name="rope_chunk_2k", op="rope", tokens=2048, hq=24, hkv=4, d=256, rot=64, off=0, inter=False,
             scaling="linear", far=1000000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "weights", "evict", "rope"])
    hkv, g, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([128, 256])
    if op == "step":
        hi = _log(rng, 64, 32768)
        batch = max(1, min(_log(rng, 1, 64), (1 << 19) // hi))
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d if batch * hi * hkv < (1 << 21) else 128,
                    lo=max(8, int(hi * rng.uniform(0.05, 1.0))), hi=hi, new=rng.choice([1, 1, 1, 2, 3, 5]))
    if op == "weights":
        tokens = _log(rng, 1, 2048)
        return dict(op=op, tokens=tokens, history=_log(rng, 1, 30720) - 1, hq=min(24, hkv * g) // hkv * hkv, hkv=hkv, d=d)
    if op == "evict":
        hi = _log(rng, 128, 32768)
        batch = max(1, min(_log(rng, 1, 64), (1 << 19) // hi))
        keep = max(16, int(hi * rng.uniform(0.08, 1.0)) - 1)
        return dict(op=op, batch=batch, hkv=hkv, d=d if batch * hi * hkv < (1 << 21) else 128,
                    lo=max(8, int(hi * rng.uniform(0.1, 1.0))), hi=hi, keep=keep, sink=rng.randrange(0, 5),
                    recent=rng.randrange(0, keep // 2))
    d = rng.choice([64, 80, 96, 128, 192, 256])
    off = rng.choice([0, 0, 0, d // 2])
    return dict(op=op, tokens=_log(rng, 1, 2048), hq=hkv * min(g, 4), hkv=hkv, d=d, rot=(d - off) // rng.choice([1, 1, 2]),
                off=off, inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]), far=_log(rng, 2048, 4000000))


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


def _inv_freq(case):
    """Rotary frequencies (fp64) and the factor on cos and sin."""
    r, base = case["rot"], 1.0e6
    inv = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if case["scaling"] == "linear":
        return inv / 4.0, 1.0
    if case["scaling"] == "yarn":
        factor, length = 8.0, 16384.0
        at = lambda turns: r * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64, device="cuda") - low) / max(high - low, 1e-3)).clamp(0, 1)
        return inv / factor * ramp + inv * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return inv, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    op, s = case["op"], dict(case)
    if op in ("step", "evict"):
        lens = _lens(case)
        order = torch.randperm(len(lens), generator=gen, device="cuda").tolist()
        lens = [lens[i] for i in order]
        s["table"], blocks = _table(gen, lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["max_ctx"] = max(lens)
        s |= _cache(gen, blocks, case["hkv"], case["d"])
        b, hkv, stride = case["batch"], case["hkv"], s["table"].shape[1] * PAGE
        # what earlier queries gave each key, on a coarse grid so that ties occur; older keys are at lower positions
        s["acc"] = torch.randn((b, hkv, stride), generator=gen, device="cuda").mul_(1.5).exp_().to(torch.bfloat16).float()
        s["slot_pos"] = torch.arange(stride, dtype=torch.int32, device="cuda").expand(b, hkv, stride).contiguous()
    if op == "step":
        b, n, hq, hkv, d = (case[x] for x in ("batch", "new", "hq", "hkv", "d"))
        s["q"], s["k_new"], s["v_new"] = _bf16(gen, b, n, hq, d), _bf16(gen, b, n, hkv, d), _bf16(gen, b, n, hkv, d)
        s["pos"] = s["lens"] + 1000  # the sequence has forgotten a thousand tokens before
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty((b, n, hq, d), dtype=torch.float32, device="cuda")
    elif op == "weights":
        n, hq, hkv, d = (case[x] for x in ("tokens", "hq", "hkv", "d"))
        s["table"], blocks = _table(gen, [case["history"] + n])
        s |= _cache(gen, blocks, hkv, d)
        s["q"], s["scale"] = _bf16(gen, n, hq, d), 1.0 / math.sqrt(d)
        s["acc"] = torch.zeros((hkv, s["table"].shape[1] * PAGE), dtype=torch.float32, device="cuda")
    elif op == "evict":
        s["acc_out"] = torch.zeros((b, hkv, case["keep"]), dtype=torch.float32, device="cuda")
        s["pos_out"] = torch.zeros((b, hkv, case["keep"]), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros_like(s["lens"])
    elif op == "rope":
        n, hq, hkv, d = (case[x] for x in ("tokens", "hq", "hkv", "d"))
        # the projection's output, q | k | v of a token side by side
        qkv = _bf16(gen, n, hq + 2 * hkv, d)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["pos"] = torch.randint(0, case["far"], (1,), generator=gen, device="cuda", dtype=torch.int32) + \
            torch.arange(n, dtype=torch.int32, device="cuda") * (1 if n > 64 else 977)
        s["inv"], s["factor"] = _inv_freq(case)
        # the plan: each frequency in turns per position, as a 64-bit fraction
        turns = (s["inv"].cpu().numpy() / (2 * math.pi) * 2.0 ** 64).round().astype(np.uint64)
        s["phases"] = torch.from_numpy(turns.view(np.int64)).cuda()
        s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty((n, hkv, d), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def _rows(s, table):
    """K rows of each sequence's pages, dequantised: [B][Hkv][keys][D]."""
    page = table.clamp(min=0).long()
    k = s["k"][page].float() * s["ks"][page][:, :, :, None, :, None]
    b, m, hkv, dc = k.shape[:4]
    return k.permute(0, 2, 1, 4, 3, 5).reshape(b, hkv, m * PAGE, dc * 16)


def _v_rows(s, table):
    page = table.clamp(min=0).long()
    v = s["v"][page].float() * s["vs"][page][:, :, :, None, :]
    b, m, hkv, d = v.shape[:4]
    return v.permute(0, 2, 1, 4, 3).reshape(b, hkv, m * PAGE, d)


def _plain_step(s):
    b, n, hq, hkv, d = s["batch"], s["new"], s["hq"], s["hkv"], s["d"]
    g, dev = hq // hkv, "cuda"
    # the new tokens' rows into their slots, their weight from zero
    slot = (s["lens"].long()[:, None] - n + torch.arange(n, device=dev)).clamp(min=0)
    page, at = s["table"].long().gather(1, slot // PAGE), slot % PAGE
    kc, kscale = _quantise(s["k_new"].float())
    vc, vscale = _quantise(s["v_new"].float())
    s["k"][page, :, :, at] = kc.view(b, n, hkv, d // 16, 16)
    s["v"][page, :, :, at] = vc
    s["ks"][page, :, at], s["vs"][page, :, at] = kscale, vscale
    bi = torch.arange(b, device=dev)[:, None]
    s["acc"][bi, :, slot] = 0.0
    s["slot_pos"][bi, :, slot] = (s["pos"][:, None] + torch.arange(n, dtype=torch.int32, device=dev))[:, :, None]
    k, v = _rows(s, s["table"]), _v_rows(s, s["table"])
    q = s["q"].float().view(b, n, hkv, g, d).transpose(1, 2).reshape(b, hkv, n * g, d)
    sc = (q @ k.transpose(2, 3)) * s["scale"]
    last = s["lens"].long()[:, None] - n + torch.arange(n, device=dev)
    seen = torch.arange(k.shape[2], device=dev) <= last.repeat_interleave(g, 1)[:, None, :, None]
    p = (sc - sc.masked_fill(~seen, -math.inf).amax(3, keepdim=True)).exp().masked_fill(~seen, 0.0)
    p = p / p.sum(3, keepdim=True)
    s["acc"] += p.sum(2)
    s["out"].copy_((p @ v).view(b, hkv, n, g, d).transpose(1, 2).reshape(b, n, hq, d))
    return [s["out"], s["acc"], s["k"], s["v"], s["ks"], s["vs"], s["slot_pos"]]


def _plain_weights(s):
    n, hq, hkv, d, hist = s["tokens"], s["hq"], s["hkv"], s["d"], s["history"]
    k = _rows(s, s["table"])[0]
    q = s["q"].float().view(n, hkv, hq // hkv, d).transpose(0, 1).reshape(hkv, -1, d)
    sc = (q @ k.transpose(1, 2)) * s["scale"]
    row = torch.arange(n, device="cuda").repeat_interleave(hq // hkv)
    hidden = torch.arange(k.shape[1], device="cuda") > hist + row[:, None]
    sc.masked_fill_(hidden, -math.inf)
    p = sc.sub_(sc.amax(2, keepdim=True)).exp_()
    p /= p.sum(2, keepdim=True)
    s["acc"] += p.sum(1, dtype=torch.float64).float()
    return [s["acc"]]


def _plain_evict(s):
    b, hkv, keep = s["batch"], s["hkv"], s["keep"]
    acc, pos, lens = s["acc"], s["slot_pos"], s["lens"].long()[:, None, None]
    t = torch.arange(acc.shape[2], device="cuda")
    live = (t < lens).expand_as(acc)
    newest = pos.masked_fill(~live, -1).amax(2, keepdim=True)
    key = acc.masked_fill((pos < s["sink"]) | (pos > newest - s["recent"]), math.inf).masked_fill(~live, -1.0)
    rank = torch.empty_like(key, dtype=torch.int64)
    rank.scatter_(2, key.sort(dim=2, descending=True, stable=True).indices, t.expand_as(acc).contiguous())
    kept = live & (rank < keep)
    new = lens.clamp(max=keep)
    # kept slots past the budget move, in order, into the slots below it that are given up
    hb, hh, ht = (~kept & (t < new)).nonzero(as_tuple=True)
    mb, mh, mt = (kept & (t >= new)).nonzero(as_tuple=True)
    sp, dp = s["table"].long()[mb, mt // PAGE], s["table"].long()[hb, ht // PAGE]
    so, do = mt % PAGE, ht % PAGE
    s["k"][dp, hh, :, do] = s["k"][sp, mh, :, so]
    s["v"][dp, hh, :, do] = s["v"][sp, mh, :, so]
    s["ks"][dp, hh, do], s["vs"][dp, hh, do] = s["ks"][sp, mh, so], s["vs"][sp, mh, so]
    n = min(keep, acc.shape[2])
    left = (t[:n] < new).expand(b, hkv, n)
    s["acc_out"][:, :, :n] = torch.where(left, acc[:, :, :n], s["acc_out"][:, :, :n])
    s["pos_out"][:, :, :n] = torch.where(left, pos[:, :, :n], s["pos_out"][:, :, :n])
    s["acc_out"][hb, hh, ht], s["pos_out"][hb, hh, ht] = acc[mb, mh, mt], pos[mb, mh, mt]
    s["new_lens"].copy_(new[:, 0, 0])
    return [s["acc_out"], s["pos_out"], s["new_lens"], s["k"], s["v"], s["ks"], s["vs"]]


def _plain_rope(s):
    r, off = s["rot"], s["off"]
    ang = s["pos"].double()[:, None] * s["inv"]
    c, sn = ((f(ang) * s["factor"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    for x, y in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        x = x.float()
        part = x[..., off:off + r]
        a, b = (part[..., 0::2], part[..., 1::2]) if s["inter"] else (part[..., :r // 2], part[..., r // 2:])
        lo, hi = a * c - b * sn, b * c + a * sn
        z = torch.stack((lo, hi), -1).flatten(-2) if s["inter"] else torch.cat((lo, hi), -1)
        y.copy_(torch.cat((x[..., :off], z, x[..., off + r:]), -1))
    return [s["q_out"], s["k_out"]]


def _own(s):
    import int8_kv_cache_quant_gb300 as kvq
    op = s["op"]
    if op == "rope":
        kvq.kvq_rope_bf16(s["q"], s["k"], s["pos"], s["phases"],
                          layout=kvq.ROPE_INTERLEAVED if s["inter"] else kvq.ROPE_HALF, rotary_offset=s["off"],
                          attn_factor=s["factor"], q_out=s["q_out"], k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    if "cache" not in s:  # the handle and the workspace that a program keeps
        s["cache"] = kvq.KVCache.wrap(s["k"], s["v"], s["ks"], s["vs"])
        if op == "step":
            need = kvq.kvq_step_accum_workspace_bytes(s["batch"], s["new"], s["hq"], s["max_ctx"], s["d"])
        elif op == "weights":
            need = kvq.kvq_chunk_weights_workspace_bytes(s["tokens"], s["hq"], s["hkv"], s["history"], s["d"])
        else:
            need = kvq.kvq_evict_workspace_bytes(s["batch"], s["hkv"], s["max_ctx"], s["keep"])
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    if op == "step":
        kvq.kvq_decode_step_accum_int8kv(s["cache"], s["k_new"], s["v_new"], s["q"], s["table"], s["lens"], s["max_ctx"],
                                         s["scale"], s["acc"], slot_pos=s["slot_pos"], pos=s["pos"], out=s["out"],
                                         workspace=s["ws"])
        return [s["out"], s["acc"], s["k"], s["v"], s["ks"], s["vs"], s["slot_pos"]]
    if op == "weights":
        kvq.kvq_attn_chunk_weights_int8kv(s["cache"], s["q"], s["history"], s["table"][0], s["scale"], s["acc"],
                                          workspace=s["ws"])
        return [s["acc"]]
    kvq.kvq_cache_evict(s["cache"], s["table"], s["lens"], s["max_ctx"], s["keep"], s["acc"], s["slot_pos"],
                        n_sink=s["sink"], n_recent=s["recent"], acc_out=s["acc_out"], slot_pos_out=s["pos_out"],
                        new_lens=s["new_lens"], workspace=s["ws"])
    return [s["acc_out"], s["pos_out"], s["new_lens"], s["k"], s["v"], s["ks"], s["vs"]]


def run(s):
    if own:
        return _own(s)
    return {"step": _plain_step, "weights": _plain_weights, "evict": _plain_evict, "rope": _plain_rope}[s["op"]](s)


# ------------------------------------------------------------------------------------ what a pass needs
def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op == "step":
        keys, n, hq, b = sum(_lens(case)), case["new"], case["hq"], case["batch"]
        # K, V and both scales of every key once, its weight read and written, the new rows, q and the output
        return dict(bytes=keys * hkv * (2 * d + 8 + 8) + b * n * (hq * d * 6 + hkv * (6 * d + 12)) + keys / 4,
                    flops=4.0 * keys * n * hq * d)
    if op == "weights":
        n, hist, hq = case["tokens"], case["history"], case["hq"]
        pairs = n * hist + n * (n + 1) / 2
        # K and its scale once, the weights read and written, q; one product of the queries with the keys they see
        return dict(bytes=(n + hist) * hkv * (d + 4 + 8) + n * hq * d * 2, flops=2.0 * pairs * hq * d)
    if op == "evict":
        size = 0.0
        for n in _lens(case):
            keep = min(n, case["keep"])
            # kept slots past the budget: the recent ones and a share of the others
            recent = min(case["recent"], n - keep)
            moves = min(keep, n - keep, recent + (keep - min(keep, case["recent"])) * (n - keep) / n)
            # weight and position of every slot read, those kept written, the moved rows read and written
            size += hkv * (n * 8 + keep * 8 + moves * 2 * (2 * d + 8))
        return dict(bytes=size, flops=0.0)
    n, heads = case["tokens"], case["hq"] + hkv
    return dict(bytes=n * heads * d * 4 + n * 4, flops=3.0 * n * heads * case["rot"])


# ------------------------------------------------------------------------------------ by the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        r, off, base = case["rot"], case["off"], np.float64(1.0e6)
        j = np.arange(r // 2)
        inv, factor = np.exp(-2.0 * j / r * np.log(base)), 1.0
        if case["scaling"] == "linear":
            inv = inv / 4.0
        elif case["scaling"] == "yarn":
            turns_dim = [r * np.log(16384.0 / (t * 2 * np.pi)) / (2 * np.log(base)) for t in (32.0, 1.0)]
            low, high = max(np.floor(turns_dim[0]), 0.0), min(np.ceil(turns_dim[1]), r - 1.0)
            mix = np.clip((j - low) / max(high - low, 1e-3), 0.0, 1.0)
            inv, factor = inv * (mix / 8.0 + (1.0 - mix)), 1.0 + 0.1 * np.log(8.0)
        turn = s["pos"].cpu().numpy().astype(np.float64)[:, None] * inv
        z = torch.from_numpy(factor * np.exp(1j * turn)).cuda()[:, None, :]
        outs = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            i = torch.arange(r // 2, device="cuda")
            ia, ib = (off + 2 * i, off + 2 * i + 1) if case["inter"] else (off + i, off + i + r // 2)
            w = torch.complex(y[..., ia], y[..., ib]) * z
            y[..., ia], y[..., ib] = w.real, w.imag
            outs.append(y)
        return outs
    if op == "evict":
        acc, pos = s["acc"].cpu().numpy(), s["slot_pos"].cpu().numpy()
        table, lens, keep = s["table"].cpu().numpy(), s["lens"].cpu().numpy(), case["keep"]
        ao = s["acc_out"].cpu().numpy().astype(np.float64)
        ks, vs = s["ks"].cpu().numpy().astype(np.float64), s["vs"].cpu().numpy().astype(np.float64)
        for b in range(case["batch"]):
            n = int(lens[b])
            new = min(n, keep)
            for h in range(case["hkv"]):
                a, p = acc[b, h, :n], pos[b, h, :n]
                guarded = (p < case["sink"]) | (p > p.max() - case["recent"])
                order = np.lexsort((np.arange(n), -a, ~guarded))  # guarded first, heavy first, low slot first
                chosen = np.zeros(n, bool)
                chosen[order[:new]] = True
                to, frm = np.nonzero(~chosen[:new])[0], new + np.nonzero(chosen[new:])[0]
                ao[b, h, :new] = a[:new]
                ao[b, h, to] = a[frm]
                for t in (ks, vs):
                    t[table[b, to // PAGE], h, to % PAGE] = t[table[b, frm // PAGE], h, frm % PAGE]
        return [ao, None, None, None, None, ks, vs]
    if op == "weights":
        n, hq, hkv, d, hist = (case[x] for x in ("tokens", "hq", "hkv", "d", "history"))
        g, keys = hq // hkv, n + hist
        acc = s["acc"].double()
        page, at = s["table"][0].long().repeat_interleave(PAGE)[:keys], torch.arange(keys, device="cuda") % PAGE
        tri = torch.arange(keys, device="cuda")[None] > hist + torch.arange(n, device="cuda")[:, None]
        for h in range(hkv):
            k = s["k"][page, h, :, at].reshape(keys, d).double() * s["ks"][page, h, at].double()[:, None]
            for j in range(g):
                z = s["q"][:, h * g + j].double() @ k.T / math.sqrt(d)
                acc[h, :keys] += torch.softmax(z.masked_fill_(tri, -math.inf), 1).sum(0)
        return [acc]
    # step
    b, n, hq, hkv, d = (case[x] for x in ("batch", "new", "hq", "hkv", "d"))
    g = hq // hkv
    out, acc = torch.zeros((b, n, hq, d), dtype=torch.float64, device="cuda"), s["acc"].double()
    ks, vs = s["ks"].double(), s["vs"].double()
    for i in range(b):
        ctx = int(s["lens"][i])
        t = torch.arange(ctx, device="cuda")
        page, at = s["table"][i].long()[t // PAGE], t % PAGE
        k = s["k"][page, :, :, at].reshape(ctx, hkv, d).double() * s["ks"][page, :, at].double()[..., None]
        v = s["v"][page, :, :, at].double() * s["vs"][page, :, at].double()[..., None]
        for rows, new, scales in ((k, s["k_new"][i], ks), (v, s["v_new"][i], vs)):
            x = new.double()
            # the codes are defined by fp32 quotients: a tie of those goes to the even code
            unit = (x.abs().amax(-1, keepdim=True).float() / torch.full((1,), 127.0, device="cuda")).double()
            rows[ctx - n:] = (x / unit).float().round().double() * unit
            scales[page[ctx - n:], :, at[ctx - n:]] = x.abs().amax(-1) / 127.0
        acc[i, :, ctx - n:ctx] = 0.0
        for j in range(n):
            m = ctx - n + 1 + j
            q = s["q"][i, j].double().view(hkv, g, d)
            p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k[:m]) / math.sqrt(d), 2)
            acc[i, :, :m] += p.sum(1)
            out[i, j] = torch.einsum("hgt,thd->hgd", p, v[:m]).reshape(hq, d)
    return [out, acc, None, None, ks, vs, None]
