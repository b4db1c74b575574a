"""The operators for long contexts on the GPU against binary64 references (tests/long_ref.py), with tolerances
from the roundings each one makes."""
import numpy as np
import pytest

import attn_ref as R
import long_ref as L
from test_gpu_attn import Batch, cu, host, rnd, tt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_amd as q
    return q


def e5m2_raw(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def i32(x):
    import torch
    return cu(x, torch.int32)


class Long(Batch):
    """A ragged batch with its bounds, scores, selections and shared prefixes."""

    def bounds(self, max_new=None, fill=0xA5, fresh=None):
        import torch
        nb = self.kvc.desc.n_blocks
        raw = torch.full((nb, self.kv, 2, self.d), fill, dtype=torch.uint8, device="cuda")
        b = raw.view(torch.float8_e5m2)
        start = self.start if fresh is None else np.concatenate([[0], np.cumsum(fresh)])
        news = self.news if fresh is None else np.array(fresh)
        self.stq.stq_kv_bounds(self.kvc, i32(self.table), i32(start), i32(self.lens), b,
                               max(1, int(news.max())) if max_new is None else max_new)
        torch.cuda.synchronize()
        return b

    def all_bounds(self):
        """Of every block, as the prompts' writes leave them."""
        return self.bounds(fill=0x7F, fresh=np.maximum(self.lens, 0))

    def score(self, b, scale=None, max_new=None, max_len=None, q=None, fill=7.0):
        import torch
        q = self.q if q is None else q
        s = torch.full((self.tok, self.kv, self.table.shape[1]), fill, device="cuda")
        self.scale = self.d ** -0.5 if scale is None else scale
        self.stq.stq_kv_score(self.kvc, b, i32(self.table), i32(self.start), i32(self.lens), q, s, self.scale,
                              max(1, int(self.news.max())) if max_new is None else max_new,
                              max(1, int(self.lens.max())) if max_len is None else max_len)
        torch.cuda.synchronize()
        return s

    def blocks(self, sel, q=None, o=None, max_new=None, scale=None):
        import torch
        stq = self.stq
        q = self.q if q is None else q
        o = torch.full_like(q, 5.0) if o is None else o
        max_new = max(1, int(self.news.max())) if max_new is None else max_new
        self.scale = self.d ** -0.5 if scale is None else scale
        n = len(self.lens)
        size = stq.stq_kv_attend_blocks_bytes(self.kvc, n, self.tok, self.heads, sel.shape[2], max_new)
        work = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
        stq.stq_kv_attend_blocks(self.kvc, i32(self.table), i32(self.start), i32(self.lens), sel, q, o, self.scale, max_new, work)
        torch.cuda.synchronize()
        return o

    def check_blocks(self, o, sel, rows=None):
        img, o, q = self.pages.cpu().numpy(), host(o), host(self.q)
        sel = sel.cpu().numpy()
        g, cols = self.heads // self.kv, self.table.shape[1]
        for i, (n, m) in enumerate(zip(self.lens, self.news)):
            n = int(min(n, cols * self.T))
            K, V, there = self.cache.request(self.table[i], n, img)
            for j in range(m):
                t = self.start[i] + j
                if rows is not None and j >= rows:
                    assert (o[t] == 5).all()
                    continue
                for h in range(self.heads):
                    listed = [b for b in sel[t, h // g] if 0 <= b < cols]
                    want, bound = L.attend_listed(q[t, h], K[:, h // g], V[:, h // g], there, n - m + j, listed, self.T, self.scale, self.dtype)
                    got = o[t, h]
                    assert np.array_equal(np.isnan(got), np.isnan(want)), (i, j, h)
                    ok = ~np.isnan(want)
                    assert (np.abs(got - want)[ok] <= bound[ok]).all(), (i, j, h, np.abs(got - want).max())
        assert (o[self.start[-1]:] == 5).all()

    def share(self, sizes, prefix):
        """Requests in groups of `sizes` (the first at request 0) share prefix[g] tokens: the first one's blocks."""
        self.groups, self.prefix = np.concatenate([[0], np.cumsum(sizes)]), np.array(prefix)
        for s, e, p in zip(self.groups, self.groups[1:], self.prefix):
            for i in range(s + 1, e):
                self.table[i, : p // self.T] = self.table[s, : p // self.T]

    def shared(self, max_own=None, max_prefix=None, q=None, o=None, max_new=None, groups=None, prefix=None):
        import torch
        stq = self.stq
        groups, prefix = self.groups if groups is None else groups, self.prefix if prefix is None else prefix
        q = self.q if q is None else q
        o = torch.full_like(q, 5.0) if o is None else o
        max_new = max(1, int(self.news.max())) if max_new is None else max_new
        max_own = max(1, int(self.lens.max())) if max_own is None else max_own
        max_prefix = int(max(list(prefix) + [0])) if max_prefix is None else max_prefix
        self.scale = self.d ** -0.5
        size = stq.stq_kv_attend_shared_bytes(self.kvc, len(self.lens), self.tok, self.heads, len(prefix), max_new, max_own, max_prefix)
        work = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        stq.stq_kv_attend_shared(self.kvc, i32(self.table), i32(self.start), i32(self.lens), i32(groups), i32(prefix), q, o,
                                 self.scale, max_new, max_own, max_prefix, work)
        torch.cuda.synchronize()
        return o


# ---------------------------------------------------------------- bounds

@pytest.mark.parametrize("T,kv,d", [(32, 1, 64), (64, 3, 128), (128, 5, 64), (256, 2, 128), (32, 2, 128)])
def test_bounds(stq, T, kv, d):
    """Blocks that hold new tokens and no others; requests without any; a table entry outside the cache; more new
    tokens than max_new or than the request has."""
    lens = [1, 0, T, T + 1, 3 * T - 5, 2 * T + 7, 517, 9, 5 * T]
    news = [1, 0, 1, 1, 2 * T + 3, 0, 517, 12, 2]
    x = Long(stq, lens, news, kv, kv, d, T, "bf16", seed=T + d)
    x.table[8, 4] = x.kvc.desc.n_blocks
    img = x.pages.cpu().numpy()
    for max_new in (int(max(news)), 3):
        got = e5m2_raw(x.bounds(max_new=max_new))
        want = {}
        for i, (n, m) in enumerate(zip(lens, news)):
            K, _, _ = x.cache.request(x.table[i], n, img)
            for c in L.touched(n, m, T, x.table.shape[1], max_new):
                if 0 <= x.table[i, c] < x.kvc.desc.n_blocks:
                    want[int(x.table[i, c])] = K[c * T: min((c + 1) * T, n)]
        assert want
        for b in range(x.kvc.desc.n_blocks):
            for h in range(kv):
                if b in want:
                    assert np.array_equal(L.e5m2_values(got[b, h]), L.bounds(want[b][:, h])), (b, h)
                else:
                    assert (got[b, h] == 0xA5).all(), (b, h)


@pytest.mark.parametrize("d", [64, 128])
def test_bounds_of_every_exponent_and_of_poison(stq, d):
    """Keys whose scales run over all exponents, tiny ones among them (E5M2 has fewer bits there: outward), and a
    poisoned key, whose block and head alone get NaN."""
    import torch
    rng = np.random.default_rng(d)
    T, kv, n = 64, 2, 40 * 64 - 9
    x = Long(stq, [n], [n], kv, kv, d, T, "bf16", seed=1)
    k = rng.standard_normal((n, kv, d)) * 2.0 ** np.repeat(rng.integers(-26, 13, (40, 1, d // 32)), 64, 0)[:n].repeat(32, -1)
    k[:, 0, 5] = np.abs(k[:, 0, 5])
    k[:, 1, 7] = -np.abs(k[:, 1, 7])
    k[130, 1, 3] = np.inf
    pos = np.arange(n)
    slots = x.table[0, pos // T] * T + pos % T
    v = np.zeros_like(k)
    stq.stq_kv_store(x.kvc, cu(slots), cu(k, torch.float32), cu(v, torch.float32))
    got = e5m2_raw(x.bounds())
    K, _, _ = x.cache.request(x.table[0], n, x.pages.cpu().numpy())
    for c in range(40):
        for h in range(kv):
            want = L.bounds(K[c * T: min((c + 1) * T, n), h])
            assert np.array_equal(L.e5m2_values(got[x.table[0, c], h]), want, equal_nan=True), (c, h)
    assert np.isnan(L.e5m2_values(got[x.table[0, 2], 1])).all() and not np.isnan(L.e5m2_values(got[x.table[0, 2], 0])).any()


# ----------------------------------------------------------------- score

def check_score(x, b, s, q=None, rows=None, fill=7.0):
    bv, s, q = L.e5m2_values(e5m2_raw(b)), host(s), host(x.q if q is None else q)
    g = x.heads // x.kv
    for i, (n, m) in enumerate(zip(x.lens, x.news)):
        n = int(min(max(n, 0), x.table.shape[1] * x.T))
        for j in range(m):
            t, p = x.start[i] + j, n - m + j
            nb = min(p // x.T + 1, x.table.shape[1]) if p >= 0 and (rows is None or j < rows) else 0
            for h in range(x.kv):
                ids = x.table[i, :nb]
                on = (ids >= 0) & (ids < bv.shape[0])
                B = bv[np.where(on, ids, 0), h]
                z = float(np.float32(x.scale)) * q[t, h * g: (h + 1) * g]
                want, size = L.score(z, B) if nb else (np.zeros(0), np.zeros(0))
                bound = L.score_bound(z, B, size) if nb else np.zeros(0)
                got = s[t, h, :nb]
                assert (got[~on] == -np.inf).all()
                nan = np.isnan(want) & on
                assert np.isnan(got[nan]).all()
                ok = on & ~nan
                assert (np.abs(got - want)[ok] <= bound[ok]).all(), (i, j, h, np.abs(got - want)[ok].max())
                assert (s[t, h, nb:] == fill).all(), (i, j, h)
    assert (s[x.start[-1]:] == fill).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,d,T,news", [
    (4, 4, 128, 32, [1, 1, 1, 1]), (8, 2, 128, 64, [1, 0, 1, 1]), (6, 2, 64, 32, [3, 1, 2, 3]), (32, 2, 128, 32, [1, 2, 1, 1]),
    (40, 2, 64, 32, [1, 1, 3, 0]), (5, 1, 128, 32, [2, 1, 9, 4]), (8, 2, 64, 128, [40, 1, 77, 5]), (2, 2, 128, 32, [100, 0, 31, 7]),
    (70, 2, 128, 32, [5, 1, 1, 2]), (16, 1, 64, 64, [33, 1, 18, 2])])
def test_score(stq, dtype, heads, kv, d, T, news):
    x = Long(stq, [600, 33, 900, 64], news, heads, kv, d, T, dtype, seed=heads, pad=2, extra_cols=2)
    b = x.all_bounds()
    x.table[2, 1], x.table[0, 0] = -1, x.kvc.desc.n_blocks + 3
    s = x.score(b)
    check_score(x, b, s)
    for max_len in (1, 100000):                            # the split of the work is not the result's
        assert (host(x.score(b, max_len=max_len)) == host(s)).all()
    check_score(x, b, x.score(b, max_new=2), rows=2)
    check_score(x, b, x.score(b, scale=-3.7e-3))


def test_score_of_hard_numbers(stq):
    """Queries of any finite size and scales that bring them back, zero scales, poisoned blocks, strided rows, requests
    with more queries than tokens."""
    import torch
    x = Long(stq, [300, 70, 3], [2, 1, 5], 8, 2, 128, 32, "bf16", seed=3)
    b = x.all_bounds()
    wide = torch.zeros(x.tok, 12, 128, dtype=x.q.dtype, device="cuda")
    base = host(x.q)
    for mag, scale in ((1.0, 0.0), (2.0 ** 120, 2.0 ** -100), (2.0 ** -120, 2.0 ** 100), (2.0 ** -126, 3e38), (1.0, -0.0)):
        wide[:, 2:10] = cu(base * mag, torch.float64).to(wide.dtype)
        q = wide[:, 2:10]
        s = x.score(b, scale=scale, q=q)
        check_score(x, b, s, q=q)
    bad = e5m2_raw(b).copy()
    bad[x.table[0, 3], 1] = 0x7F
    bb = cu(bad).view(torch.float8_e5m2)
    s = x.score(bb)
    assert np.isnan(host(s)[0, 1, 3]) and not np.isnan(host(s)[0, 0]).any()
    check_score(x, bb, s)


# ---------------------------------------------------------------- select

def run_select(stq, s, lens, news, T, k, first, last, max_new=None, pad=0):
    import torch
    start = np.concatenate([[0], np.cumsum(news)])
    sel = torch.full((s.shape[0], s.shape[1], k), -7, dtype=torch.int32, device="cuda")
    stq.stq_kv_select(cu(s, torch.float32), i32(start), i32(lens), sel, T, max(1, max(news)) if max_new is None else max_new, first, last)
    torch.cuda.synchronize()
    return sel.cpu().numpy(), start


@pytest.mark.parametrize("cols", [1, 5, 63, 64, 65, 128, 129, 500, 512, 513, 2048, 2049, 8192, 8200, 32768])
@pytest.mark.parametrize("k,first,last", [(1, 0, 0), (4, 1, 2), (64, 0, 1), (130, 3, 0), (7, 3, 4)])
def test_select(stq, cols, k, first, last):
    """Against choosing one by one: equal scores, NaN, infinities, zeros of both signs, fewer blocks than asked for."""
    T, kv = 32, 2
    rng = np.random.default_rng(cols + k)
    lens = [cols * T, max(1, cols * T // 2), min(cols * T, 70), 5]
    news = [2, 1, 0, 6]
    s = rng.standard_normal((sum(news) + 1, kv, cols)).astype(np.float32)
    s[1] = np.round(s[1] * 2) / 2                          # many are equal
    s[2, 0] = 3.25
    odd = rng.integers(0, cols, (3, cols // 6 + 1))
    s[0, 0, odd[0]], s[0, 0, odd[1]], s[1, 1, odd[2]] = np.nan, -np.inf, np.inf
    s[1, 0, ::3], s[1, 0, 1::3] = 0.0, -0.0
    s[2, 1] = -np.abs(s[2, 1])
    got, start = run_select(stq, s, lens, news, T, k, first, last)
    for i, (n, m) in enumerate(zip(lens, news)):
        for j in range(m):
            for h in range(kv):
                t = start[i] + j
                assert got[t, h].tolist() == L.select(s[t, h], n - m + j, T, k, first, last), (i, j, h)
    assert (got[-1] == -7).all()


def test_select_rows(stq):
    """Rows of many requests, past max_new and behind the last one; a number of rows that fills no workgroup."""
    rng = np.random.default_rng(3)
    T, kv, cols = 64, 3, 40
    lens, news = rng.integers(1, cols * T, 33), rng.integers(0, 5, 33)
    s = np.round(rng.standard_normal((int(news.sum()) + 3, kv, cols)) * 8).astype(np.float32)
    for max_new in (None, 2):
        got, start = run_select(stq, s, lens, list(news), T, 9, 1, 1, max_new)
        for i, (n, m) in enumerate(zip(lens, news)):
            for j in range(m):
                for h in range(kv):
                    t = start[i] + j
                    want = [-7] * 9 if max_new is not None and j >= max_new else L.select(s[t, h], n - m + j, T, 9, 1, 1)
                    assert got[t, h].tolist() == want, (i, j, h)
        assert (got[start[-1]:] == -7).all()


# ---------------------------------------------------------------- blocks

def lists(x, k, rng, odd=True):
    """Random lists: some short, some with entries that stand for nothing, one empty, one with a block twice."""
    cols = x.table.shape[1]
    sel = np.full((x.tok, x.kv, k), -1)
    for t in range(x.tok):
        for h in range(x.kv):
            n = min(k, cols, int(rng.integers(1, k + 1)))
            at = np.sort(rng.choice(k, n, replace=False)) if odd else np.arange(n)
            sel[t, h, at] = np.sort(rng.choice(cols, n, replace=False))
    if odd:
        sel[0, 0] = -1
        sel[-1, -1, 0] = cols + 5
        sel[x.tok // 2, 0, -1] = 2 ** 31 - 1
        if k > 1:
            sel[x.tok // 3, 0, :2] = 0
    return i32(sel)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,d,T,news,k", [
    (4, 4, 128, 32, [1, 1, 1, 1], 3), (8, 2, 128, 64, [1, 0, 1, 1], 5), (6, 2, 64, 32, [3, 1, 2, 3], 9), (32, 2, 128, 32, [1, 2, 1, 1], 4),
    (40, 2, 64, 128, [1, 1, 3, 0], 2), (70, 2, 128, 32, [5, 1, 1, 2], 7), (5, 1, 128, 256, [2, 1, 9, 4], 1), (8, 2, 64, 32, [40, 1, 17, 5], 6)])
def test_blocks(stq, dtype, heads, kv, d, T, news, k):
    x = Long(stq, [700, 33, 900, 64], news, heads, kv, d, T, dtype, seed=heads, pad=2, extra_cols=1)
    x.table[2, 1] = -1
    sel = lists(x, k, np.random.default_rng(k))
    x.check_blocks(x.blocks(sel), sel)
    if max(news) > 2:
        x.check_blocks(x.blocks(sel, max_new=2), sel, rows=2)


@pytest.mark.parametrize("dtype,heads,kv,d,T,k,n", [("bf16", 8, 2, 128, 64, 70, 1), ("fp16", 4, 1, 64, 32, 130, 2), ("bf16", 20, 1, 128, 32, 90, 1),
                                                    ("bf16", 8, 8, 128, 32, 33, 16), ("fp16", 4, 4, 128, 256, 12, 3)])
def test_blocks_long_lists(stq, dtype, heads, kv, d, T, k, n):
    """Lists long enough that their work is split or taken by sixteen waves."""
    x = Long(stq, [k * T * 5 // 4] * n, [1] * n, heads, kv, d, T, dtype, seed=k)
    sel = lists(x, k, np.random.default_rng(k))
    x.check_blocks(x.blocks(sel), sel)


def test_blocks_of_everything_is_attention(stq):
    """All blocks listed, in any order: what stq_kv_attend computes, to its own bound."""
    import torch
    x = Long(stq, [900, 31, 400], [3, 1, 2], 8, 2, 128, 32, "bf16", seed=2)
    cols = x.table.shape[1]
    sel = i32(np.stack([[np.random.default_rng(t).permutation(cols)] * 2 for t in range(x.tok)]))
    o = x.blocks(sel)
    x.check(o)
    q = x.q.clone()
    assert torch.equal(x.blocks(sel, q=q, o=q), o)           # in place


def test_blocks_poisoned_and_strided(stq):
    """A poisoned key reaches the queries whose list and position reach it, no other; strided rows."""
    import torch
    x = Long(stq, [128, 96], [2, 1], 4, 2, 64, 32, "fp16", seed=8)
    k = torch.full((1, 2, 64), float("nan"), device="cuda")
    k[:, 1] = 0.5
    stq.stq_kv_store(x.kvc, cu([x.table[0, 2] * 32 + 5]), k, torch.zeros_like(k))
    sel = i32([[[0, 2, 3], [0, 2, 3]], [[0, 1, 3], [0, 1, 2]], [[0, 1, 2], [2, -1, 0]]])
    o = x.blocks(sel)
    assert np.isnan(host(o)[0, :2]).all() and not np.isnan(host(o)[0, 2:]).any() and not np.isnan(host(o)[1:]).any()
    x.check_blocks(o, sel)
    wide = torch.zeros(x.tok, 9, 64, dtype=x.q.dtype, device="cuda")
    wide[:, 3:7] = x.q
    out = torch.full((x.tok, 6, 64), 5.0, dtype=x.q.dtype, device="cuda")
    x.blocks(sel, q=wide[:, 3:7], o=out[:, 1:5])
    assert torch.equal(torch.nan_to_num(out[:, 1:5]), torch.nan_to_num(o)) and (out[:, 0] == 5).all() and (out[:, 5] == 5).all()


# ---------------------------------------------------------------- shared

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,d,T,sizes,prefix,new", [
    (8, 2, 128, 64, [3, 1, 2], [192, 64, 0], 1), (4, 4, 64, 32, [5], [96], 1), (8, 1, 128, 32, [9, 2], [320, 32], 2),
    (16, 4, 64, 64, [4, 4], [128, 256], 3), (32, 2, 128, 32, [2, 3], [224, 96], 1), (8, 2, 128, 32, [2, 2], [96, 160], 40),
    (6, 2, 64, 32, [3, 3], [96, 32], 30), (40, 2, 128, 32, [12], [352], 1), (8, 2, 64, 32, [20, 20], [352, 288], 1)])
def test_shared(stq, dtype, heads, kv, d, T, sizes, prefix, new):
    """Groups of several sizes, one that shares nothing, requests in no group; few rows and many on either side."""
    rng = np.random.default_rng(heads + new)
    lens, news = [], []
    for s, p in zip(sizes, prefix):
        for i in range(s):
            news.append(new if i == 0 else int(rng.integers(0, new + 1)))
            lens.append(p + news[-1] + int(rng.integers(0, 90)))
    lens += [70, 33]                                         # in no group
    news += [1, 1]
    x = Long(stq, lens, news, heads, kv, d, T, dtype, seed=new, pad=2)
    x.share(sizes, prefix)
    for max_own, max_prefix in ((None, None), (1, 1), (100000, 100000)):
        x.check(x.shared(max_own=max_own, max_prefix=max_prefix))


def test_shared_prefix_past_the_first_new_token(stq):
    """A prefix that is no whole number of blocks, or that reaches into a member's new tokens, is cut; members without
    new tokens do not cut it; negative ones share nothing."""
    x = Long(stq, [200, 130, 300, 64], [1, 40, 2, 0], 8, 2, 128, 32, "bf16", seed=4)
    x.share([4], [128])
    x.table[1, 3] = x.table[0, 3]
    for p in (128, 90, 127, 70, 31, 0, -5, 100000):
        if p == 100000:                                      # (only what the rows of the table agree in may be claimed)
            x.table[2, :9] = x.table[0, :7].tolist() + x.table[2, 7:9].tolist()
        x.check(x.shared(prefix=[p], max_prefix=128))


def test_shared_blocks_outside_the_cache(stq):
    x = Long(stq, [300, 290, 310], [1, 2, 1], 8, 2, 128, 32, "bf16", seed=5)
    x.share([3], [256])
    x.table[:, 3], x.table[:, 0] = -1, x.kvc.desc.n_blocks
    x.check(x.shared())
    x.table[1, 8:] = -1                                      # nothing of its own but the prefix
    x.check(x.shared())
    x.table[:, :] = -1                                       # nothing at all
    assert (host(x.shared()) == 0).all()


def test_shared_many_groups(stq):
    """More groups than a wave has lanes, some empty; a call without groups."""
    import torch
    n = 150
    rng = np.random.default_rng(6)
    x = Long(stq, rng.integers(66, 140, n), [1] * n, 4, 2, 64, 32, "bf16", seed=6)
    sizes = [2] * 70 + [0] * 9 + [3, 1, 0, 2]
    x.share(sizes, [64] * len(sizes))
    o = x.shared()
    x.check(o)
    x.check(x.shared(groups=[0], prefix=[]))
    q = x.q.clone()
    assert torch.equal(x.shared(q=q, o=q), o)                # in place


def test_shared_larger_than_a_tile(stq):
    """Rows of a group over several tiles of the prompt kernel, prefixes over many parts, rows past max_new."""
    x = Long(stq, [1100] * 40 + [900] * 9, [4] * 40 + [9] * 9, 8, 1, 128, 64, "bf16", seed=7)
    x.share([40, 9], [1024, 832])
    x.check(x.shared(max_own=128))
    x.check(x.shared(max_own=128, max_new=3), rows=3)


# -------------------------------------------------------------- together

class Step:
    """A layer's step over long contexts: plan, cache write, bounds, scores, selection, attention over the selection,
    and the same tokens' attention behind a shared prefix, in buffers of its own."""

    def __init__(self, stq, n, heads, kv, d, T, blocks, cols, tok, k, max_new):
        import torch
        z = dict(device="cuda")
        i = torch.int32
        self.stq, self.n, self.k, self.max_new = stq, n, k, max_new
        self.pages = torch.full((stq.stq_kv_bytes(blocks, T, kv, d),), 0xFF, dtype=torch.uint8, **z)
        self.kvc = stq.make_kv(self.pages, T, kv, d)
        self.heads, self.T = heads, T
        self.bounds = torch.full((blocks, kv, 2, d), 0x7F, dtype=torch.uint8, **z).view(torch.float8_e5m2)
        self.table = torch.full((n, cols), -1, dtype=i, **z)
        self.free = torch.arange(blocks, dtype=i, **z)
        self.cached, self.new = torch.zeros(n, dtype=i, **z), torch.zeros(n, dtype=i, **z)
        self.start, self.lens, self.used = torch.zeros(n + 1, dtype=i, **z), torch.zeros(n, dtype=i, **z), torch.zeros(1, dtype=i, **z)
        self.pos, self.slots = torch.zeros(tok, dtype=i, **z), torch.zeros(tok, dtype=torch.int64, **z)
        self.qkv = torch.zeros(tok, heads + 2 * kv, d, dtype=torch.bfloat16, **z)
        self.score = torch.zeros(tok, kv, cols, **z)
        self.sel = torch.full((tok, kv, k), -7, dtype=i, **z)
        self.o, self.os = (torch.zeros(tok, heads, d, dtype=torch.bfloat16, **z) for _ in range(2))
        self.group, self.prefix = torch.tensor([0, n], dtype=i, **z), torch.zeros(1, dtype=i, **z)
        w1 = stq.stq_kv_attend_blocks_bytes(self.kvc, n, tok, heads, k, max_new)
        w2 = stq.stq_kv_attend_shared_bytes(self.kvc, n, tok, heads, 1, max_new, cols * T, cols * T)
        self.w1 = torch.zeros(w1, dtype=torch.uint8, **z) if w1 else None
        self.w2 = torch.zeros(w2, dtype=torch.uint8, **z)
        self.scale, self.kv, self.cols = d ** -0.5, kv, cols

    def step(self):
        s, m = self.stq, self.max_new
        s.stq_kv_plan(self.cached, self.new, self.free, self.table, self.T, self.kvc.desc.n_blocks, self.start, self.lens, self.pos,
                      self.slots, self.used)
        q, k, v = self.qkv[:, :self.heads], self.qkv[:, self.heads:self.heads + self.kv], self.qkv[:, self.heads + self.kv:]
        s.stq_kv_store(self.kvc, self.slots, k, v)
        s.stq_kv_bounds(self.kvc, self.table, self.start, self.lens, self.bounds, m)
        s.stq_kv_score(self.kvc, self.bounds, self.table, self.start, self.lens, q, self.score, self.scale, m, self.cols * self.T)
        s.stq_kv_select(self.score, self.start, self.lens, self.sel, self.T, m, 1, 1)
        s.stq_kv_attend_blocks(self.kvc, self.table, self.start, self.lens, self.sel, q, self.o, self.scale, m, self.w1)
        s.stq_kv_attend_shared(self.kvc, self.table, self.start, self.lens, self.group, self.prefix, q, self.os, self.scale, m,
                               self.cols * self.T, self.cols * self.T, self.w2)


ROUNDS = ([100, 70, 68], [1, 1, 1], [3, 0, 2], [1, 40, 1], [1, 1, 1])


def rounds(rng, tok):
    cached = np.zeros(3, int)
    for new in ROUNDS:
        raw = rnd(rng, (tok, 12, 128), "bf16") + cu(np.repeat(rng.standard_normal((tok // 14 + 1, 12, 128)), 14, 0)[:tok], tt("bf16"))
        yield cached, new, raw
        cached = cached + np.array(new)


def feed(X, cached, new, raw):
    import torch
    X.qkv.copy_(raw)
    X.cached.copy_(i32(cached))
    X.new.copy_(i32(new))
    X.o.fill_(1.0)
    X.os.fill_(1.0)
    X.free.copy_(i32(np.roll(np.arange(X.free.numel()), -getattr(X, "freed", 0))))


def test_together(stq):
    """Prompts, then tokens: every step's selection is that of the bounds of what the cache holds, its output the
    attention over it; the blocks of the selection hold the largest logits' bounds; behind a shared prefix of
    nothing the output is that of stq_kv_attend."""
    import torch
    X = Step(stq, 3, 8, 2, 128, 32, 64, 14, 240, 4, 128)
    rng = np.random.default_rng(5)
    X.freed = 0
    for cached, new, raw in rounds(rng, 240):
        feed(X, cached, new, raw)
        X.step()
        torch.cuda.synchronize()
        X.freed += int(X.used.item())
        table, lens, start = X.table.cpu().numpy(), X.lens.cpu().numpy(), X.start.cpu().numpy()
        cache = R.Cache(64, 32, 2, 128)
        img = X.pages.cpu().numpy()
        bv, sel, s = L.e5m2_values(e5m2_raw(X.bounds)), X.sel.cpu().numpy(), host(X.score)
        q, o, os_ = host(X.qkv)[:, :8], host(X.o), host(X.os)
        for i in range(3):
            K, V, there = cache.request(table[i], int(lens[i]), img)
            assert there.all()
            for c in range(-(-lens[i] // 32)):
                for h in range(2):
                    assert np.array_equal(bv[table[i, c], h], L.bounds(K[32 * c: 32 * c + 32, h]))
            for t in range(start[i], start[i + 1]):
                p = int(lens[i]) - int(start[i + 1]) + t
                for h in range(8):
                    sc = s[t, h // 4]
                    assert sel[t, h // 4].tolist() == L.select(sc, p, 32, 4, 1, 1)
                    logits = X.scale * (K[: p + 1, h // 4] @ q[t, h])
                    top = np.array([logits[32 * c: 32 * c + 32].max() for c in range(p // 32 + 1)])
                    assert (sc[: top.size] >= top - 1e-3 * (1 + np.abs(top))).all()
                    want, bound = L.attend_listed(q[t, h], K[:, h // 4], V[:, h // 4], there, p, sel[t, h // 4], 32, X.scale, "bf16")
                    assert (np.abs(o[t, h] - want) <= bound).all()
                    want, bound = L.attend_listed(q[t, h], K[:, h // 4], V[:, h // 4], there, p, range(14), 32, X.scale, "bf16")
                    assert (np.abs(os_[t, h] - want) <= bound).all()
        assert (o[start[-1]:] == 1).all() and (os_[start[-1]:] == 1).all()


def test_together_in_a_graph(stq):
    """The seven calls captured once and replayed over changing buffers, with eager work and synchronisations
    between, give what eager calls give, bit for bit; so do calls on a stream of their own."""
    import torch
    rng = np.random.default_rng(9)
    args = (stq, 3, 8, 2, 128, 32, 64, 14, 240, 4, 128)
    A, B, C = Step(*args), Step(*args), Step(*args)
    A.step()
    torch.cuda.synchronize()
    A.table.fill_(-1)
    A.bounds.view(torch.uint8).fill_(0x7F)
    A.pages.fill_(0xFF)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.step()
    other = torch.cuda.Stream()
    freed = 0
    for r, (cached, new, raw) in enumerate(rounds(rng, 240)):
        for X in (A, B, C):
            X.freed = freed
            feed(X, cached, new, raw)
            X.prefix.fill_(32 * (r % 2))                     # (request 0's first block is not the others': see below)
            X.group.copy_(i32([0, 1]))                       # a group of one request
        torch.cuda.synchronize()
        g.replay()
        B.step()
        with torch.cuda.stream(other):
            C.step()
        torch.cuda.synchronize()
        for name in ("o", "os", "table", "lens", "start", "pos", "slots", "used", "sel", "score", "pages"):
            for X in (B, C):
                assert torch.equal(getattr(A, name), getattr(X, name)), (r, name)
        for X in (B, C):
            assert torch.equal(A.bounds.view(torch.uint8), X.bounds.view(torch.uint8))
        freed += int(A.used.item())
        torch.ones(1000, device="cuda").sum().item()


def test_blocks_of_many_tokens(stq):
    """Token and head pairs enough for a wave each."""
    for dtype, heads, kv, d, T in (("bf16", 8, 4, 128, 32), ("fp16", 4, 4, 64, 64)):
        x = Long(stq, [700, 40], [520, 3], heads, kv, d, T, dtype, seed=d, extra_cols=1)
        x.table[0, 2] = -1
        sel = lists(x, 5, np.random.default_rng(d))
        x.check_blocks(x.blocks(sel), sel)


@pytest.mark.parametrize("heads,kv,d,news", [(4, 2, 128, [20, 1]), (2, 2, 64, [70, 3]), (12, 2, 64, [17, 17]), (8, 2, 128, [2, 1])])
def test_score_of_long_requests(stq, heads, kv, d, news):
    """More blocks than a wave's window of the table, over several parts of the work."""
    x = Long(stq, [32 * 701, 32 * 300 + 5], news, heads, kv, d, 32, "bf16", seed=d)
    b = x.all_bounds()
    x.table[0, 300:310] = -1
    s = x.score(b)
    check_score(x, b, s)
    assert (host(x.score(b, max_len=50)) == host(s)).all()


def test_shared_more_requests_than_lanes(stq):
    """Past 256 requests what the workgroups know of the batch is looked up another way; the result is the same."""
    rng = np.random.default_rng(11)
    for new, prefix in ((1, [128, 0, 96]), (9, [128, 64, 96])):
        sizes = [200, 3, 90]
        lens = np.concatenate([p + new + rng.integers(0, 40, s) for s, p in zip(sizes, prefix)])
        x = Long(stq, lens, [new] * 293, 8, 1, 64, 32, "bf16", seed=new)
        x.share(sizes, prefix)
        o = x.shared()
        x.check(o)


def test_long_contexts_past_32_bits(stq):
    """Blocks more than 4 GiB into the cache give what the first ones give, bit for bit."""
    import torch
    T, kv, d = 256, 8, 128
    x = Long(stq, [900, 256, 513], [3, 1, 40], 16, kv, d, T, "bf16", seed=12)
    x.share([3], [256])
    small, nb = x.kvc, x.kvc.desc.n_blocks
    sel = lists(x, 3, np.random.default_rng(1), odd=False)
    b = x.all_bounds()
    want = (x.score(b), x.blocks(sel), x.shared())
    at = (5 << 30) // (x.pages.numel() // nb)
    big = torch.zeros((at + nb) * (x.pages.numel() // nb), dtype=torch.uint8, device="cuda")
    big[at * (x.pages.numel() // nb):] = x.pages.flatten()
    x.kvc = stq.make_kv(big, T, kv, d)
    x.table = np.where(x.table >= 0, x.table + at, -1)
    bb = x.all_bounds()
    assert torch.equal(bb[at:].view(torch.uint8), b.view(torch.uint8)) and (e5m2_raw(bb[:at]) == 0x7F).all()
    for a, c in zip(want, (x.score(bb), x.blocks(sel), x.shared())):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(c))
    assert small.desc.n_blocks == nb


def test_calls_of_slices(stq):
    """Requests a .. b-1 of a plan in a call of their own: the same rows, the others left alone."""
    import torch
    x = Long(stq, [300, 64, 500, 33], [2, 1, 30, 1], 8, 2, 128, 32, "bf16", seed=13)
    b = x.all_bounds()
    s = x.score(b)
    sel = lists(x, 4, np.random.default_rng(2), odd=False)
    o, c = x.blocks(sel), x.shared(groups=[0], prefix=[])
    i, n = torch.int32, 4
    table, start, lens = i32(x.table), i32(x.start), i32(x.lens)
    s2, o2, c2 = torch.full_like(s, 7.0), torch.full_like(o, 5.0), torch.full_like(c, 5.0)
    for lo, hi, new in ((0, 2, 2), (2, 3, 30), (3, 4, 1)):
        t, st, le = table[lo:hi], start[lo:hi + 1], lens[lo:hi]
        stq.stq_kv_score(x.kvc, b, t, st, le, x.q, s2, x.scale, new, 500)
        w = stq.stq_kv_attend_blocks_bytes(x.kvc, hi - lo, x.tok, 8, 4, new)
        stq.stq_kv_attend_blocks(x.kvc, t, st, le, sel, x.q, o2, x.scale, new, torch.empty(w, dtype=torch.uint8, device="cuda") if w else None)
        w = stq.stq_kv_attend_shared_bytes(x.kvc, hi - lo, x.tok, 8, 0, new, 500, 0)
        stq.stq_kv_attend_shared(x.kvc, t, st, le, torch.zeros(1, dtype=i, device="cuda"), torch.zeros(0, dtype=i, device="cuda"), x.q, c2,
                                 x.scale, new, 500, 0, torch.empty(w, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert n == len(x.lens)
    check_score(x, b, s2)
    x.check_blocks(o2, sel)
    x.check(c2)
