"""Plain binary64 references of the softmax layers' operators, from their
formulas (include/stq.h); shares no code with the library."""
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E_MIN, E_MAX = -23, 13
# half a rounding step relative to the value
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def block_exp(m):
    """Least e in [-23, 13] with m <= 6 * 2^e; 0 for m = 0."""
    if m == 0:
        return 0
    e = E_MIN
    while e < E_MAX and m > 6 * 2.0 ** e:
        e += 1
    return e


def quantise(x):
    """Codes and exponents of x [..., d], channel by channel search over the levels."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    b = x.reshape(-1, d // 32, 32)
    e = np.vectorize(block_exp, otypes=[np.int64])(np.abs(b).max(-1))
    a = np.minimum(np.abs(b) / 2.0 ** e[..., None].astype(np.float64), 6.0)    # saturation
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])            # even codes first: they take the ties
    code = order[np.abs(a[..., None] - LEVELS[order]).argmin(-1)]
    code = np.where(np.signbit(b), code + 8, code)          # a zero keeps its sign
    return code.reshape(x.shape).astype(np.uint8), e.reshape(x.shape[:-1] + (d // 32,))


def value(code, e):
    """Values of codes [..., d] with exponents [..., d/32]."""
    mag = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    return mag * np.repeat(2.0 ** np.asarray(e, np.float64), 32, -1)


class Cache:
    """The cache's bytes on the host: [block][head] of key codes, value codes, key scales, value scales."""

    def __init__(self, n_blocks, T, heads, d, fill=0):
        self.n_blocks, self.T, self.heads, self.d = n_blocks, T, heads, d
        self.raw = np.full((n_blocks, heads, T * d * 17 // 16), fill, np.uint8)

    def parts(self, img=None):
        r = self.raw if img is None else np.asarray(img).reshape(self.raw.shape)
        T, d = self.T, self.d
        c = T * d // 2
        s = T * d // 32
        nb, h = r.shape[:2]
        return (r[..., :c].reshape(nb, h, T, d // 2), r[..., c:2 * c].reshape(nb, h, T, d // 2),
                r[..., 2 * c:2 * c + s].reshape(nb, h, d // 32, T), r[..., 2 * c + s:].reshape(nb, h, d // 32, T))

    def store(self, slots, k, v):
        kc, vc, ks, vs = self.parts()
        for t, s in enumerate(np.asarray(slots)):
            if s < 0 or s >= self.n_blocks * self.T:
                continue
            b, o = int(s) // self.T, int(s) % self.T
            for h in range(self.heads):
                kk, vv = np.asarray(k[t, h], np.float64), np.asarray(v[t, h], np.float64)
                bad = not (np.isfinite(kk).all() and np.isfinite(vv).all())
                if bad:
                    kk, vv = np.zeros_like(kk), np.zeros_like(vv)
                for x, code, sc in ((kk, kc, ks), (vv, vc, vs)):
                    c, e = quantise(x)
                    code[b, h, o] = c[0::2] | (c[1::2] << 4)
                    sc[b, h, :, o] = e + 127
                if bad:
                    ks[b, h, :, o] = 255

    def values(self, slot, img=None):
        """(keys, values) [heads][d] in binary64 at one token slot."""
        kc, vc, ks, vs = self.parts(img)
        b, o = int(slot) // self.T, int(slot) % self.T
        out = []
        for code, sc in ((kc, ks), (vc, vs)):
            by = code[b, :, o]
            c = np.stack([by & 15, by >> 4], -1).reshape(self.heads, self.d)
            s = sc[b, :, :, o].astype(np.int64)
            x = value(c, np.where(s == 255, 0, s - 127))
            out.append(np.where(np.repeat(s == 255, 32, -1), np.nan, x))
        return out

    def request(self, row, length, img=None):
        """Keys and values [length][heads][d] of one request's table row; a
        token of a block outside the cache is None-like: NaN with seen = False."""
        K = np.zeros((length, self.heads, self.d))
        V = np.zeros_like(K)
        there = np.zeros(length, bool)
        for s in range(length):
            b = int(row[s // self.T])
            if 0 <= b < self.n_blocks:
                K[s], V[s] = self.values(b * self.T + s % self.T, img)
                there[s] = True
        return K, V, there


def plan(cached, new, free, table, T, n_blocks, n_tok):
    """The plan, one block and one token at a time."""
    table = np.array(table, copy=True)
    cols = table.shape[1]
    used, start = 0, [0]
    pos, slot = [], []
    for i, (c, m) in enumerate(zip(cached, new)):
        c, m = max(int(c), 0), max(int(m), 0)
        for col in range(-(-c // T), min(-(-(c + m) // T), cols)):
            table[i, col] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + m):
            blk = int(table[i, p // T]) if p // T < cols else -1
            pos.append(p)
            slot.append(blk * T + p % T if 0 <= blk < n_blocks else -1)
        start.append(start[-1] + m)
    pad = max(0, n_tok - len(pos))
    lens = [max(int(c), 0) + max(int(m), 0) for c, m in zip(cached, new)]
    return dict(table=table, tok_start=np.array(start), lens=np.array(lens), pos=np.array(pos + [-1] * pad)[:n_tok],
                slots=np.array(slot + [-1] * pad)[:n_tok], used=np.array([used]))


def norm_rope(x, norm, eps, w, pos, table, n_rot, adjacent):
    """x [tokens][heads][d] -> (y, size): size bounds what binary32 roundings are relative to."""
    y = np.asarray(x, np.float64)
    d = y.shape[-1]
    if norm:
        ss = (y ** 2).sum(-1, keepdims=True)
        y = y / np.sqrt((ss / d if norm == 1 else ss) + float(np.float32(eps)))
    if w is not None:
        y = y * np.asarray(w, np.float64)
    out, size = y.copy(), np.abs(y)
    if n_rot:
        h = n_rot // 2
        cs = np.asarray(table, np.float64)[np.asarray(pos)][:, None]
        c, s = cs[..., :h], cs[..., h:]
        ia = np.arange(0, n_rot, 2) if adjacent else np.arange(h)
        ib = ia + 1 if adjacent else ia + h
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia], size[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return out, size


def norm_bound(out, size, d, out_type):
    """One rounding of the result; before it the sum of d squares (a chain of 8
    and a tree of at most 5 more: 13 roundings, halved by the root), eps, root,
    quotient, two products and the rotation's product and sum: at most 16
    binary32 half steps of the terms.  A binary16 result below 2^-14 is off by up
    to half its smallest step, 2^-25."""
    return HALF[out_type] * np.abs(out) * 1.001 + 16 * 2.0 ** -24 * size + (2.0 ** -25 if out_type == "fp16" else 2.0 ** -126)


def attend(q, K, V, there, base, scale, window, sink, out_type):
    """One head: q [rows][d] at positions base + row, K, V [length][d].
    Returns (o, bound).

    The bound: cached values and queries enter the products exactly (scaled by
    a power of two), d products summed in binary32 by steps that may truncate:
    d * 2^-23 of sum |q k|; the logit's scaling 2 half steps of its own size and
    the reference's; exp2 within 2 steps (2^-22); the weight rounded to
    binary16: 2^-11 of itself, or 2^-25 of the row's largest weight where it is
    subnormal there (2^-24 with a truncating conversion).  The sum takes
    the same rounded weights, so each moves o by its share of v - o.  Sums of
    len terms in binary32, in chains of at most len/32 + 40 steps."""
    q, K, V = (np.asarray(a, np.float64) for a in (q, K, V))
    L = K.shape[0]
    o = np.zeros((q.shape[0], V.shape[1]))
    bound = np.zeros_like(o)
    for r in range(q.shape[0]):
        p = base + r
        s = np.arange(L)
        see = (s <= p) & there
        if window:
            see &= (s > p - window) | (s < sink)
        if not see.any():
            continue
        k, v = K[see], V[see]
        logit = scale * (k @ q[r])
        if not np.isfinite(logit).all():
            o[r] = np.nan
            continue
        size = abs(scale) * (np.abs(k) @ np.abs(q[r]))
        w = np.exp(logit - logit.max())
        tot = w.sum()
        o[r] = (w[:, None] * v).sum(0) / tot
        d = q.shape[1]
        err = d * 2.0 ** -23 * (size + size.max()) + 4 * 2.0 ** -24 * (np.abs(logit) + np.abs(logit).max()) + 2.0 ** -21 + 2.0 ** -10
        away = np.abs(v - o[r])
        steps = (L / 32 + 40) * 2.0 ** -23
        bound[r] = (((err * w + 2.0 ** -24)[:, None] * away).sum(0) + steps * (w[:, None] * (np.abs(v) + np.abs(o[r]))).sum(0)) / tot
        bound[r] += HALF[out_type] * np.abs(o[r]) * 1.001 + 2.0 ** -25
    return o, bound
