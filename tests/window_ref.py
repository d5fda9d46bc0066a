"""Plain references (numpy) of the operators around windowed attention: rotary positions with several axes and the
append with rotation.  They read the documented layouts and share no code with the library."""
import numpy as np

PAGE = 16


def sections_to_axes(sections, order):
    """The axis of each frequency."""
    if order == "chunked":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def turns(pos, phases, axis_of):
    """Turns [T][r/2] as signed 64-bit fractions: the product with the position modulo 2^64."""
    p = np.asarray(pos, np.int64)[np.array(list(axis_of))].T.astype(np.uint64)
    with np.errstate(over="ignore"):
        return (p * np.asarray(phases, np.uint64)).astype(np.int64)


def angles(pos, phases, axis_of):
    return turns(pos, phases, axis_of).astype(np.float64) * (2 * np.pi / 2.0 ** 64)


def cos_sin_f32(t, factor):
    """factor cos and factor sin of the turns to the nearest fp32, through the longest float there is."""
    a = t.astype(np.longdouble) * (2 * np.longdouble("3.14159265358979323846264338327950288") / np.longdouble(2.0) ** 64)
    f = np.longdouble(np.float32(factor))
    return (np.cos(a) * f).astype(np.float32), (np.sin(a) * f).astype(np.float32)


def rotate_f32(x, c, s, off, inter):
    """x [T][H][D] fp32 rotated with the header's roundings."""
    y = x.copy()
    half = c.shape[1]
    i = np.arange(half)
    ia, ib = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + half + i)
    c, s = c[:, None], s[:, None]
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def quantise(x):
    """The rule on fp32 rows: (codes, scales)."""
    amax = np.abs(x).max(-1).astype(np.float32)
    scale = (amax / np.float32(127.0)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = (x / scale[..., None]).astype(np.float32)
    code = np.clip(np.rint(np.where(amax[..., None] > 0, q, 0.0)), -127, 127).astype(np.int8)
    return code, scale


def append(pool, k, v, seq, slot, table):
    """Rows k, v [T][Hkv][D] fp32 into a forget_ref.Pool's pages; which tokens were written."""
    (kc, ks), (vc, vs) = quantise(k), quantise(v)
    done = []
    for i in range(len(seq)):
        ok = 0 <= seq[i] < table.shape[0] and 0 <= slot[i] < PAGE * table.shape[1]
        page = int(table[seq[i], slot[i] // PAGE]) if ok else -1
        ok = ok and 0 <= page < pool.nb
        done.append(ok)
        if ok:
            at = slot[i] % PAGE
            pool.k[page, :, :, at] = kc[i].reshape(pool.hkv, pool.d // 16, 16)
            pool.v[page, :, :, at] = vc[i]
            pool.ks[page, :, at], pool.vs[page, :, at] = ks[i], vs[i]
    return np.array(done)


def attend(k, v, ok, q, pos, window, sink, scale):
    """Attention of rows q [R][D] at positions pos [R] over keys k, v [n][D] (0 .. n-1, ok: on a page of the pool), 64 bits:
    out [R][D], the bound of the relative error of a weight (as forget_ref.weights derives it) and mag = sum p |v|."""
    n, D = k.shape
    t, p = np.arange(n)[None], np.asarray(pos, np.int64)[:, None]
    seen = (t <= p) & ((t > p - window) | (t < sink)) & ok[None]
    s = np.where(seen, (q @ k.T) * scale, -np.inf)
    m = s.max(1, keepdims=True, initial=-np.inf)
    w = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = w.sum(1, keepdims=True)
    w = w / np.where(l > 0, l, 1.0)
    amp = (np.abs(q) @ np.abs(k).T * scale * 1.4427 * seen).max(1, initial=0.0)
    rel = 4 * np.log(2) * amp * (D / 16 + 5) * 2.0 ** -23 + 4 * 2.0 ** -22 + seen.sum(1) * 2.0 ** -24
    return w @ v, rel, w @ np.abs(v)


def unread_pages(table, lens, n_new, window, sink, fill):
    """The block tables with every entry that no row sees replaced by `fill`."""
    t = table.copy()
    for b, n in enumerate(lens):
        low = max(0, int(n) - n_new - window + 1) // PAGE
        t[b, -(-sink // PAGE):low] = fill
    return t


def prompt(pool, table_row, q, history, window, sink, scale):
    """Windowed attention of the queries q [T][Hq][D] (fp64 of bf16), 64 bits: out [T][Hq][D], and what an fp32 result of the
    tensor-core kernel may be off.

    A weight is 2^(z - r), z = S kf + lv with S the exact products' fp32 sum (16 a step, at most a step of 2^-23 of the
    partial sums each), kf = k_scale c two roundings, lv = log2 v_scale two steps, z and z - r one rounding each: with A
    the largest c sum |q k| and B the largest |z|, |dz| <= A (D / 16 + 5) 2^-23 + 4 B 2^-24; twice that times ln 2 for the weight
    and its sum, two exponentials of 2^-22, the additions of the sum (n 2^-24), quotient and inverse scale.  In the
    numerator it is rounded to fp16, half a step: 2^-11 relative, or 2^-25 absolute where the largest weight of the row
    is at least 1: 2^-25 max(p v_scale) sum |code| in the output."""
    T, Hq, D = q.shape
    n = history + T
    k, v, ok = pool.rows(table_row, n)
    G = Hq // pool.hkv
    page, at = np.where(ok, np.asarray(table_row)[np.arange(n) // PAGE], 0), np.arange(n) % PAGE
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    t, p = np.arange(n)[None], (history + np.arange(T))[:, None]
    seen = (t <= p) & ((t > p - window) | (t < sink)) & ok[None]
    for h in range(Hq):
        kh, vh = k[h // G], v[h // G]
        vs = pool.vs[page, h // G, at].astype(np.float64)
        code = np.abs(vh) / np.where(vs > 0, vs, 1.0)[:, None]
        s = np.where(seen, (q[:, h] @ kh.T) * scale, -np.inf)
        m = s.max(1, keepdims=True, initial=-np.inf)
        w = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
        l = w.sum(1, keepdims=True)
        w = w / np.where(l > 0, l, 1.0)
        a = (np.abs(q[:, h]) @ np.abs(kh).T * scale * 1.4427 * seen).max(1, initial=0.0)
        b = a + np.abs(np.log2(np.maximum(vs, 2.0 ** -100))).max()
        dz = a * (D / 16 + 5) * 2.0 ** -23 + 4 * b * 2.0 ** -24
        rel = 2 * np.log(2) * dz + 4 * 2.0 ** -22 + 2 * seen.sum(1) * 2.0 ** -24
        out[:, h] = w @ vh
        tol[:, h] = (rel[:, None] + 2.0 ** -11) * (w @ np.abs(vh)) + \
            2.0 ** -25 * (w * vs).max(1, initial=0.0)[:, None] * (seen @ code) + 1e-30
    return out, tol
