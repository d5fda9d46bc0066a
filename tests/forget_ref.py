"""Plain references (numpy, fp64) of the operators around a cache that forgets: decode with
accumulated weights, chunk weights, eviction and rotary positions.  They read the documented cache
layout through numpy axes and share no code with the library."""
import numpy as np

PAGE = 16


class Pool:
    """Host copy of a paged cache: random int8 codes and scales, or the contents of a GPU cache."""

    def __init__(self, k, v, ks, vs):
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.nb, self.hkv, dc = k.shape[:3]
        self.d = dc * 16

    @classmethod
    def random(cls, rng, nb, hkv, d):
        return cls(rng.integers(-127, 128, (nb, hkv, d // 16, PAGE, 16), dtype=np.int8),
                   rng.integers(-127, 128, (nb, hkv, d, PAGE), dtype=np.int8),
                   rng.uniform(0.005, 0.03, (nb, hkv, PAGE)).astype(np.float32),
                   rng.uniform(0.005, 0.03, (nb, hkv, PAGE)).astype(np.float32))

    @classmethod
    def of(cls, cache):
        return cls(*(t.cpu().numpy().copy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))

    def copy(self):
        return Pool(self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy())

    def to_gpu(self, kvq):
        import torch
        return kvq.KVCache.wrap(*(torch.from_numpy(a.copy()).cuda() for a in (self.k, self.v, self.ks, self.vs)))

    def rows(self, table_row, n):
        """Dequantised K and V of keys 0 .. n-1: [Hkv][n][D] fp64, and which keys lie on a page of the pool."""
        t = np.arange(n)
        page = np.asarray(table_row)[t // PAGE]
        ok = (page >= 0) & (page < self.nb)
        p, s = np.where(ok, page, 0), t % PAGE
        k = self.k[p, :, :, s, :].reshape(n, self.hkv, self.d).astype(np.float64) * self.ks[p, :, s][..., None]
        v = self.v[p, :, :, s].astype(np.float64) * self.vs[p, :, s][..., None]
        return k.transpose(1, 0, 2), v.transpose(1, 0, 2), ok

    def same(self, other):
        return all(np.array_equal(a.view(np.uint8), b.view(np.uint8))
                   for a, b in ((self.k, other.k), (self.v, other.v), (self.ks, other.ks), (self.vs, other.vs)))


def weights(k, v, ok, q, limits, scale):
    """Softmax weights of one (sequence, KV head): k, v [n][D], q rows [R][D], row r sees keys
    t < limits[r] on good pages.  Returns p [R][n] (zeros for a row with no key), out [R][D], the bound
    of the relative error of a weight computed in fp32 [R], and mag = sum_t p |v| [R][D].

    The bound: a score in log2 units is c * sum_d q_d k_d with c = scale log2(e).  The products are exact
    (8-bit times 7-bit significands); the tensor core adds 16 of them a step in fp32, losing at most an
    fp32 step (2^-23) of the partial sums a step, and the two partial accumulators, the key's scale, the
    row's factor, the maximum's subtraction round (2^-24) at most five more times: |ds| <= A (D / 16 + 5)
    2^-23, A the largest c sum_d |q_d k_d|.  A weight is 2^(s - M) / l: twice 2 ln2 |ds| relative (itself
    and l), two hardware exponentials (2^-22 each, on s - M and on the split's maximum), the additions of
    l in order (n 2^-24), a product and a quotient."""
    n, D = k.shape
    s = (q @ k.T) * scale
    seen = (np.arange(n)[None] < np.asarray(limits)[:, None]) & ok[None]
    s = np.where(seen, s, -np.inf)
    m = s.max(1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = p.sum(1, keepdims=True)
    p = p / np.where(l > 0, l, 1.0)
    amp = (np.abs(q) @ np.abs(k).T * scale * 1.4427 * seen).max(1, initial=0.0)
    rel = 4 * np.log(2) * amp * (D / 16 + 5) * 2.0 ** -23 + 4 * 2.0 ** -22 + n * 2.0 ** -24
    return p, p @ v, rel, p @ np.abs(v)


def bf16(x):
    import workloads as W
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(np.asarray(x, np.float32)))


def evict(pool, table, lens, cap, keep, n_sink, n_recent, acc, pos):
    """Eviction by sorting.  Returns (pool, acc_out, pos_out of the kept slots as lists [b][h], new_lens)."""
    pool = pool.copy()
    outs, new_lens = [], []
    for b, n in enumerate(lens):
        n = max(0, min(int(n), cap))
        new = min(n, keep)
        new_lens.append(new)
        row = []
        for h in range(pool.hkv):
            a, p = acc[b, h, :n].copy(), pos[b, h, :n].copy()
            ao, po = a[:new].copy(), p[:new].copy()
            if n > keep:
                guard = (p < n_sink) | (p.astype(np.int64) > int(p.max()) - n_recent)
                val = np.where(np.isnan(a), -np.inf, a.astype(np.float64))
                order = np.lexsort((np.arange(n), np.isnan(a), -val, ~guard))
                kept = np.zeros(n, bool)
                kept[order[:keep]] = True
                dst, src = np.nonzero(~kept[:keep])[0], keep + np.nonzero(kept[keep:])[0]
                assert len(dst) == len(src)
                ao[dst], po[dst] = a[src], p[src]
                for d, s in zip(dst, src):
                    dp, sp = table[b, d // PAGE], table[b, s // PAGE]
                    if not (0 <= dp < pool.nb and 0 <= sp < pool.nb):
                        continue
                    pool.k[dp, h, :, d % PAGE] = pool.k[sp, h, :, s % PAGE]
                    pool.v[dp, h, :, d % PAGE] = pool.v[sp, h, :, s % PAGE]
                    pool.ks[dp, h, d % PAGE] = pool.ks[sp, h, s % PAGE]
                    pool.vs[dp, h, d % PAGE] = pool.vs[sp, h, s % PAGE]
            row.append((ao, po))
        outs.append(row)
    return pool, outs, np.array(new_lens, np.int32)


def inv_freq(r, base, kind="none", factor=1.0, length=0.0, low=1.0, high=32.0, divisors=None):
    """Rotary frequencies and the factor on cos and sin, by the formulas of the header."""
    j = np.arange(r // 2, dtype=np.float64)
    attn = 1.0
    if kind == "ntk":
        base = base * factor ** (r / (r - 2.0))
    inv = base ** (-2.0 * j / r)
    if kind == "linear":
        inv = inv / factor
    elif kind == "yarn":
        d = lambda n: r * np.log(length / (2 * np.pi * n)) / (2 * np.log(base))  # noqa: E731
        lo, hi = max(np.floor(d(high)), 0.0), min(np.ceil(d(low)), r - 1.0)
        m = np.clip((j - lo) / max(hi - lo, 1e-3), 0, 1)
        inv = inv / factor * m + inv * (1 - m)
        attn = 0.1 * np.log(factor) + 1.0 if factor > 1 else 1.0
    elif kind == "bands":
        m = np.clip((length * inv / (2 * np.pi) - low) / (high - low), 0, 1)
        inv = inv / factor * (1 - m) + inv * m
    elif kind == "divisors":
        inv = inv / np.asarray(divisors)
    return inv, attn


def rotate(x, ang, factor, off, inter):
    """x [T][H][D] fp64 rotated by ang [T][r/2]."""
    y = x.copy()
    half = ang.shape[1]
    i = np.arange(half)
    ia, ib = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + half + i)
    c, s = factor * np.cos(ang)[:, None], factor * np.sin(ang)[:, None]
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y
