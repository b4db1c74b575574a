"""Plain binary64 references of the operators for long contexts (include/stq.h, "LONG CONTEXTS"); shares no code
with the library."""
import numpy as np

import attn_ref as R


def e5m2(x, up):
    """The nearest E5M2 number at or above (below) each x of magnitude up to 57,344."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -14))
    step = np.ldexp(1.0, e - 3)
    return (np.ceil if up else np.floor)(x / step) * step


def e5m2_values(raw):
    """Numbers that bytes stand for, from their sign, exponent and mantissa bits."""
    b = np.asarray(raw).astype(np.int64)
    sign, e, m = np.where(b & 0x80, -1.0, 1.0), (b >> 2) & 31, b & 3
    v = np.where(e == 0, m * 2.0 ** -16, np.ldexp(1 + m / 4, e - 15))
    return sign * np.where(e == 31, np.where(m == 0, np.inf, np.nan), v)


def touched(length, new, T, cols, max_new):
    """Block columns that hold the first max_new of `new` tokens that end at `length`."""
    length = min(max(length, 0), cols * T)
    base = length - new
    end = min(base + min(new, max_new), length)
    return range(max(base, 0) // T, -(-end // T)) if end > 0 and new > 0 else range(0)


def bounds(keys):
    """keys [tokens][d] -> [2][d] (NaN where any key is)."""
    if np.isnan(keys).any():
        return np.full((2, keys.shape[1]), np.nan)
    return np.stack([e5m2(keys.min(0), False), e5m2(keys.max(0), True)])


def score(x, b):
    """x [heads][d] scaled queries, b [blocks][2][d] -> (score [blocks], size): size bounds what the roundings
    of d products' sum are relative to."""
    with np.errstate(invalid="ignore"):
        parts = np.maximum(x[:, None] * b[None, :, 0], x[:, None] * b[None, :, 1])     # [heads][blocks][d]
    parts = np.where(np.isnan(b).any((1, 2))[None, :, None], np.nan, parts)
    return parts.sum(-1).max(0), np.abs(parts).sum(-1).max(0)


def score_bound(x, b, size):
    """Products are exact: d steps of a binary32 sum that may truncate, two roundings of the result; channels of a
    query below 2^-38 of its largest may be lost to binary16's range."""
    return (x.shape[-1] * 2.0 ** -23 + 4 * 2.0 ** -24) * size + 2.0 ** -38 * np.abs(x).max() * np.abs(b).max((1, 2)) * x.shape[-1]


def select(s, p, T, n_sel, n_first, n_last):
    """Columns for one row: the always-taken ones, then one by one the best of the others."""
    nb = min(p // T + 1, len(s)) if p >= 0 else 0
    must = [b for b in range(nb) if b < n_first or b >= nb - n_last]
    rank = sorted((b for b in range(nb) if b not in set(must) and not s[b] == -np.inf),
                  key=lambda b: (0 if np.isnan(s[b]) else 1, 0.0 if np.isnan(s[b]) else -float(s[b]), b))
    took = sorted(must + rank[: max(0, n_sel - len(must))])
    return took + [-1] * (n_sel - len(took))


def attend_listed(q, K, V, there, p, listed, T, scale, out_type):
    """One query row q [d] at position p over the blocks of a list: tokens of a block that is listed m times count m
    times.  (o [d], bound [d]) by attn_ref.attend on the tokens written out."""
    at = [s for b in listed if 0 <= b * T <= p for s in range(b * T, min((b + 1) * T, p + 1, len(there))) if there[s]]
    if not at:
        return np.zeros(V.shape[1]), np.zeros(V.shape[1])
    o, bound = R.attend(q[None], K[at], V[at], np.ones(len(at), bool), len(at), scale, 0, 0, out_type)
    return o[0], bound[0]
