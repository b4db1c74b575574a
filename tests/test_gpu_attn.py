"""The softmax layers' operators on the GPU against binary64 references
(tests/attn_ref.py), with tolerances from the roundings each one makes."""
import numpy as np
import pytest

import attn_ref as R

pytestmark = pytest.mark.gpu

TYPES = ("bf16", "fp16", "fp32")


def tt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def cu(x, dtype=None):
    import torch
    return torch.as_tensor(np.asarray(x), device="cuda", dtype=dtype)


def host(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_amd as q
    return q


def rnd(rng, shape, dtype):
    return cu(rng.standard_normal(shape), tt("fp32")).to(tt(dtype))


# ----------------------------------------------------------------- store

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,heads,d", [(32, 1, 64), (64, 3, 128), (128, 2, 64), (256, 5, 128)])
def test_store_and_fetch(stq, dtype, T, heads, d):
    """Bytes equal to the definition's; strided sources; slots in any order,
    some outside the cache; untouched bytes stay; the read-back is exact."""
    import torch
    rng = np.random.default_rng(T + heads)
    n_blocks, n = 3, 41
    ref = R.Cache(n_blocks, T, heads, d, fill=0xA5)
    pages = cu(ref.raw).clone()
    both = rnd(rng, (n, 2 * heads + 1, d), dtype) * cu(np.exp(2 * rng.standard_normal((n, 1, 1))), tt("fp32")).to(tt(dtype))
    both = both.to(tt(dtype))
    k, v = both[:, 1:1 + heads], both[:, 1 + heads:]
    k[0] = 0
    v[1, :, :32] = 0
    slots = rng.permutation(n_blocks * T)[:n].astype(np.int64)
    slots[5], slots[6], slots[7] = -1, n_blocks * T, -2 ** 40
    kv = stq.make_kv(pages, T, heads, d)
    stq.stq_kv_store(kv, cu(slots), k, v)
    torch.cuda.synchronize()
    ref.store(slots, host(k), host(v))
    assert np.array_equal(pages.cpu().numpy(), ref.raw)
    for out in TYPES:
        ko = torch.full((n, heads, d), 7.0, dtype=tt(out), device="cuda")
        vo = torch.full_like(ko, 7.0)
        stq.stq_kv_fetch(kv, cu(slots), ko, vo)
        for t, s in enumerate(slots):
            if 0 <= s < n_blocks * T:
                a, b = ref.values(s)
                assert np.array_equal(host(ko[t]), a) and np.array_equal(host(vo[t]), b)
            else:
                assert (host(ko[t]) == 7).all() and (host(vo[t]) == 7).all()


def test_store_ties_extremes_and_poison(stq):
    """Every level and every midpoint at every exponent, values past both ends
    of the scale's range, subnormals; infinities and NaN poison their token
    and head alone."""
    import torch
    lev = R.LEVELS
    pts = np.concatenate([lev, (lev[1:] + lev[:-1]) / 2, np.nextafter(np.float32((lev[1:] + lev[:-1]) / 2), np.float32(9)),
                          np.nextafter(np.float32((lev[1:] + lev[:-1]) / 2), np.float32(0))]).astype(np.float32)
    pts = np.concatenate([pts, -pts, np.zeros(4, np.float32)])     # 62: what two blocks hold beside their largest
    rows = []
    for e in list(range(-30, 20)) + [-127, -140, 120]:
        blk = np.zeros(64, np.float32)
        for half in (0, 1):
            blk[32 * half] = 6
            blk[32 * half + 1: 32 * half + 32] = pts[31 * half: 31 * half + 31]
        with np.errstate(over="ignore"):
            rows.append(np.ldexp(blk, e).astype(np.float32))
    rows = np.stack(rows)
    rows = rows[np.isfinite(rows).all(1)]
    n = len(rows)
    k = np.stack([rows, rows[::-1]], 1)                   # [n][2][64]
    v = k[::-1].copy()
    bad = {3: np.inf, 7: -np.inf, 9: np.nan}
    for t, x in bad.items():
        k[t, 0, 5] = x
        v[t + 20, 1, 63] = x
    ref = R.Cache(2, 32, 2, 64)
    pages = cu(ref.raw).clone()
    kv = stq.make_kv(pages, 32, 2, 64)
    slots = np.arange(n)[:64]
    k, v = k[:64], v[:64]
    stq.stq_kv_store(kv, cu(slots), cu(k), cu(v))
    torch.cuda.synchronize()
    ref.store(slots, k, v)
    assert np.array_equal(pages.cpu().numpy(), ref.raw)
    ko, vo = torch.empty(len(k), 2, 64, device="cuda"), torch.empty(len(k), 2, 64, device="cuda")
    stq.stq_kv_fetch(kv, cu(slots), ko, vo)
    nan = np.isnan(host(ko)).all(-1)
    want = np.zeros_like(nan)
    for t in bad:
        want[t, 0] = want[t + 20, 1] = True
    assert np.array_equal(nan, want) and (host(vo)[want] == 0).all() and np.isfinite(host(ko)[~want]).all()


# ------------------------------------------------------------------ plan

def run_plan(stq, cached, new, free, table, T, n_blocks, n_tok):
    import torch
    n = len(cached)
    i = torch.int32
    t = cu(table, i)
    out = dict(table=t, tok_start=torch.full((n + 1,), -7, dtype=i, device="cuda"), lens=torch.full((n,), -7, dtype=i, device="cuda"),
               pos=torch.full((n_tok,), -7, dtype=i, device="cuda"), slots=torch.full((n_tok,), -7, dtype=torch.int64, device="cuda"),
               used=torch.full((1,), -7, dtype=i, device="cuda"))
    stq.stq_kv_plan(cu(cached, i), cu(new, i), cu(free, i), t, T, n_blocks, out["tok_start"], out["lens"], out["pos"],
                    out["slots"], out["used"])
    torch.cuda.synchronize()
    return {k: x.cpu().numpy() for k, x in out.items()}


@pytest.mark.parametrize("n,T,top,most", [(1, 32, 0, 1), (1, 256, 900, 4000), (7, 64, 300, 1), (63, 32, 100, 40), (64, 64, 500, 3),
                                          (511, 32, 64, 90), (513, 128, 700, 5), (4096, 64, 200, 3)])
def test_plan(stq, n, T, top, most):
    rng = np.random.default_rng(n + T)
    cached = rng.integers(0, top + 1, n)
    new = rng.integers(0, most + 1, n)
    new[-1] = most
    cols = -(-(top + most) // T)
    have = -(-cached // T)
    need = int((-(-(cached + new) // T) - have).sum())
    n_blocks = int(have.sum()) + need + 5
    ids = rng.permutation(n_blocks)
    table = np.full((n, cols), -9)
    at = 0
    for i in range(n):
        table[i, :have[i]] = ids[at:at + have[i]]
        at += have[i]
    tok = int(new.sum())
    for free, cap in ((ids[at:], tok), (ids[at:at + need // 2], tok + 37), (ids[at:], max(1, tok // 2))):
        got, want = run_plan(stq, cached, new, free, table, T, n_blocks, cap), R.plan(cached, new, free, table, T, n_blocks, cap)
        for k in want:
            assert np.array_equal(got[k], want[k]), k


def test_plan_odd_inputs(stq):
    """Negative counts, a table too narrow for its request, entries outside the
    cache, an empty free list, no token at all."""
    table = np.array([[3, 99, -1], [-5, 2, -1], [1, -1, -1], [0, 4, 5]])
    cached, new = [40, 70, -3, 96], [10, 1, 40, 33]
    for free in ([7, 8], [], [100, 6]):
        got, want = run_plan(stq, cached, new, free, table, 32, 10, 90), R.plan(cached, new, free, table, 32, 10, 90)
        for k in want:
            assert np.array_equal(got[k], want[k]), (free, k)
    got = run_plan(stq, [5, 6], [0, -1], [1], [[0], [1]], 32, 4, 0)
    assert got["tok_start"].tolist() == [0, 0, 0] and got["lens"].tolist() == [5, 6] and got["used"].tolist() == [0]


# ------------------------------------------------------------------ norm

def cos_sin(n_pos, n_rot):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(n_rot // 2) * 2 / n_rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


@pytest.mark.parametrize("d,n_rot", [(64, 0), (64, 16), (64, 64), (128, 32), (128, 48), (128, 128), (256, 64), (256, 256)])
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("io", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("adjacent", [0, 1])
def test_norm_rope(stq, d, n_rot, norm, io, adjacent):
    import torch
    if adjacent and not n_rot:
        pytest.skip("no rotation, no pairs")
    rng = np.random.default_rng(d + n_rot)
    n, hq, hk = 5, 7, 2
    both = rnd(rng, (n, hq + 2 * hk, d), io[0])
    both[2, 1] = 0                                         # a row of zeros
    q, k = both[:, :hq], both[:, hq:hq + hk]
    keep = both.clone()
    wq = None if norm == 0 else cu(1 + 0.3 * rng.standard_normal(d), tt("fp32"))
    wk = cu(1 + 0.3 * rng.standard_normal(d), tt("fp32"))
    table = pos = None
    if n_rot:
        table = cos_sin(4001, n_rot)
        pos = np.array([0, 4000, -1, 17, 4001])            # the third and the last row are padding
    qo = torch.full((n, hq, d), 3.0, dtype=tt(io[1]), device="cuda")
    ko = torch.full((n, hk, d), 3.0, dtype=tt(io[1]), device="cuda")
    stq.stq_qk_norm_rope(q, k, qo, ko, norm=norm, eps=1e-6, q_weight=wq, k_weight=wk,
                         pos=None if pos is None else cu(pos, torch.int32), cos_sin=None if table is None else cu(table),
                         rot_pairs=adjacent)
    torch.cuda.synchronize()
    assert torch.equal(both, keep)
    on = np.ones(n, bool) if pos is None else (pos >= 0) & (pos < 4001)
    for x, o, w in ((q, qo, wq), (k, ko, wk)):
        y, size = R.norm_rope(host(x)[on], norm, 1e-6, None if w is None else host(w), None if pos is None else pos[on], table,
                              n_rot, adjacent)
        err = np.abs(host(o)[on] - y)
        assert (err <= R.norm_bound(y, size, d, io[1])).all(), (err / R.norm_bound(y, size, d, io[1])).max()
        assert (host(o)[~on] == 3).all()


def test_norm_in_place_and_without_keys(stq):
    """In place on views of one buffer gives what separate outputs give; one
    token, one head; no keys."""
    import torch
    rng = np.random.default_rng(5)
    table, pos = cu(cos_sin(50, 128)), cu([3, 49, 0], torch.int32)
    both = rnd(rng, (3, 6, 128), "bf16")
    q, k = both[:, :4], both[:, 4:5]
    qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(3, 1, 128, dtype=q.dtype, device="cuda")
    stq.stq_qk_norm_rope(q, k, qo, ko, pos=pos, cos_sin=table)
    last = both[:, 5].clone()
    stq.stq_qk_norm_rope(q, k, q, k, pos=pos, cos_sin=table)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(both[:, 5], last)
    one = rnd(rng, (1, 1, 64), "fp32")
    out = torch.empty_like(one)
    stq.stq_qk_norm_rope(one, None, out, None, norm=stq.STQ_NORM_L2, eps=1e-6)
    y, size = R.norm_rope(host(one), 2, 1e-6, None, None, None, 0, 0)
    assert (np.abs(host(out) - y) <= R.norm_bound(y, size, 64, "fp32")).all()


# ---------------------------------------------------------------- attend

class Batch:
    """Requests over a cache whose unwritten bytes are all ones (NaN scales)."""

    def __init__(self, stq, lens, news, heads, kv, d, T, dtype, seed=0, pad=0, spare=3, extra_cols=0):
        import torch
        rng = np.random.default_rng(seed)
        self.stq, self.dtype, self.T = stq, dtype, T
        self.lens, self.news = np.array(lens), np.array(news)
        self.heads, self.kv, self.d = heads, kv, d
        need = -(-np.maximum(self.lens, 0) // T)
        cols = int(max(need.max(), 1)) + extra_cols
        nb = int(need.sum()) + spare
        ids = rng.permutation(nb)
        self.table = np.full((len(lens), cols), -1)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = ids[at:at + m]
            at += m
        self.cache = R.Cache(nb, T, kv, d, fill=0xFF)
        self.pages = cu(self.cache.raw).clone()
        self.kvc = stq.make_kv(self.pages, T, kv, d)
        prof = np.exp(0.5 * rng.standard_normal((kv, d)))
        slots = np.concatenate([self.table[i, np.arange(m) // T] * T + np.arange(m) % T for i, m in enumerate(self.lens)]
                               ).astype(np.int64)
        if len(slots):
            k = rng.standard_normal((len(slots), kv, d)) * prof
            v = rng.standard_normal((len(slots), kv, d)) * prof
            stq.stq_kv_store(self.kvc, cu(slots), cu(k, tt("fp32")), cu(v, tt("fp32")))
        self.start = np.concatenate([[0], np.cumsum(self.news)])
        self.tok = int(self.start[-1]) + pad
        self.q = rnd(rng, (self.tok, heads, d), dtype)

    def run(self, window=0, sink=0, scale=None, max_new=None, max_len=None, q=None, work=None, o=None):
        import torch
        stq = self.stq
        q = self.q if q is None else q
        o = torch.full_like(q, 5.0) if o is None else o
        max_new = max(1, int(self.news.max())) if max_new is None else max_new
        max_len = max(1, int(self.lens.max())) if max_len is None else max_len
        self.scale = self.d ** -0.5 if scale is None else scale
        i = torch.int32
        if work is None:
            size = stq.stq_kv_attend_bytes(self.kvc, len(self.lens), self.tok, self.heads, max_new, max_len, window, sink)
            work = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
        stq.stq_kv_attend(self.kvc, cu(self.table, i), cu(self.start, i), cu(self.lens, i), q, o, self.scale, max_new, max_len,
                          window, sink, work)
        torch.cuda.synchronize()
        return o

    def check(self, o, window=0, sink=0, q=None, rows=None, nan=()):
        """Every row against the reference; returns the worst error over its bound."""
        img = self.pages.cpu().numpy()
        o, q = host(o), host(self.q if q is None else q)
        g, worst = self.heads // self.kv, 0.0
        for i, (L, m) in enumerate(zip(self.lens, self.news)):
            K, V, there = self.cache.request(self.table[i], int(min(L, self.table.shape[1] * self.T)), img)
            j = np.arange(m) if rows is None else np.arange(m)[:rows]
            for h in range(self.heads):
                s = slice(self.start[i], self.start[i] + len(j))
                want, bound = R.attend(q[s, h], K[:, h // g], V[:, h // g], there, int(L) - int(m), self.scale, window, sink, self.dtype)
                got = o[s, h]
                assert np.array_equal(np.isnan(got), np.isnan(want)), (i, h)
                ok = ~np.isnan(want)
                err = np.abs(got - want)[ok]
                ratio = float((err / np.maximum(bound[ok], 1e-300)).max()) if err.size and err.max() > 0 else 0.0
                assert ratio <= 1.0, (i, h, ratio, err.max())
                worst = max(worst, ratio)
            if rows is not None:
                assert (o[self.start[i] + len(j): self.start[i + 1]] == 5).all()
        assert (o[self.start[-1]:] == 5).all()             # rows behind the last sequence
        return worst


LENS = [1, 0, 31, 32, 33, 64, 65, 200, 517]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,d,T", [(4, 4, 64, 32), (8, 2, 128, 64), (6, 1, 64, 128), (10, 2, 128, 256), (16, 1, 128, 32),
                                          (40, 2, 64, 64), (3, 3, 128, 32)])
def test_attend_single_tokens(stq, dtype, heads, kv, d, T):
    B = Batch(stq, LENS, [1] * len(LENS), heads, kv, d, T, dtype, seed=heads, pad=2, extra_cols=1)
    B.check(B.run())


@pytest.mark.parametrize("window,sink", [(1, 0), (7, 1), (32, 4), (33, 64), (100, 40), (600, 5), (64, 0)])
@pytest.mark.parametrize("d,T,news", [(64, 32, 1), (128, 64, 3), (64, 128, 40)])
def test_attend_window(stq, window, sink, d, T, news):
    lens = [1, 33, 65, 200, 517, 95]
    B = Batch(stq, lens, [min(news, 5 + 7 * i) for i in range(len(lens))], 6, 2, d, T, "bf16", seed=window)
    B.check(B.run(window, sink), window, sink)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,d", [(4, 4, 64), (8, 2, 128), (5, 1, 128), (16, 1, 64)])
@pytest.mark.parametrize("news", [[2, 0, 5, 1], [8, 3, 0, 33], [70, 129, 1, 64]])
def test_attend_many_tokens(stq, dtype, heads, kv, d, news):
    """Drafted tokens and prompts over nothing, a little and a lot that is cached."""
    B = Batch(stq, [news[0], news[1] + 40, news[2] + 300, news[3] + 7], news, heads, kv, d, 64, dtype, seed=sum(news), pad=3)
    B.check(B.run())


def test_attend_more_queries_than_tokens(stq):
    """Queries before position 0 see nothing; a request without tokens too."""
    B = Batch(stq, [3, 0, 40], [9, 4, 40], 4, 2, 64, 32, "bf16")
    o = B.run()
    B.check(o)
    assert (host(o)[:6] == 0).all() and (host(o)[9:13] == 0).all()


@pytest.mark.parametrize("lens", [[4000, 17, 2100], [5000]])
@pytest.mark.parametrize("news", [1, 4, 20])
def test_attend_split(stq, lens, news):
    """Work split over the cache and joined; the hint of the longest length
    changes the split, not the result."""
    B = Batch(stq, lens, [news] * len(lens), 8, 2, 128, 64, "fp16", seed=news)
    for hint in (None, 1, 1 << 20):
        B.check(B.run(max_len=hint))
    B.check(B.run(window=1500, sink=10), 1500, 10)


@pytest.mark.parametrize("news", [1, 3, 30])
def test_attend_split_narrow_heads(stq, news):
    """The same at d = 64, one request's length far above the stated longest."""
    B = Batch(stq, [3333, 900, 2500], [news] * 3, 6, 1, 64, 128, "bf16", seed=news)
    for hint in (None, 1100):
        B.check(B.run(max_len=hint))


@pytest.mark.parametrize("news", [30, 70])
def test_attend_many_requests(stq, news):
    """More requests than the order of the prompts' tiles is worked out for; new
    tokens and lengths ragged, some requests without any."""
    rng = np.random.default_rng(news)
    new = rng.integers(0, news + 1, 67)
    new[5], new[66], new[11] = news, news, 0
    B = Batch(stq, new + rng.integers(0, 60, 67), new, 3, 1, 64, 32, "bf16", seed=news, pad=4)
    B.check(B.run())


def test_attend_head_groups_larger_than_a_tile(stq):
    """160 query heads of one key/value head: a token's rows fill more than one tile."""
    B = Batch(stq, [300, 45, 0], [3, 1, 1], 160, 1, 64, 32, "bf16", seed=5, pad=1)
    B.check(B.run())


def test_attend_order_of_ragged_prompts(stq):
    """Up to 64 requests: every tile of every request, whatever their number and
    lengths (bands that no request's tile lies in, requests without new tokens)."""
    rng = np.random.default_rng(7)
    for n in (1, 2, 5, 23, 64):
        new = rng.integers(0, 200 if n < 10 else 50, n)
        new[-1] = 131
        old = rng.integers(0, 40, n)
        old[n // 2] += 900
        B = Batch(stq, new + old, new, 2, 1, 64, 64, "fp16", seed=n, pad=1)
        B.check(B.run(window=70, sink=3), 70, 3)


def test_offsets_past_32_bits(stq):
    """Blocks whose bytes lie past 4 GiB hold what blocks at the front hold."""
    import torch
    T, heads, d = 256, 8, 128
    one = stq.stq_kv_bytes(1, T, heads, d)
    n_blocks = (9 << 29) // one                              # 4.5 GiB
    pages = torch.empty(n_blocks * one, dtype=torch.uint8, device="cuda")
    kv = stq.make_kv(pages, T, heads, d)
    assert kv.desc.n_blocks == n_blocks
    rng = np.random.default_rng(2)
    L = 700
    k, v = rnd(rng, (L, heads, d), "bf16"), rnd(rng, (L, heads, d), "bf16")
    q = rnd(rng, (L, 16, d), "bf16")
    outs = []
    for first in (0, n_blocks - 3):
        t = np.arange(L)
        slots = cu((first + t // T) * T + t % T)
        stq.stq_kv_store(kv, slots, k, v)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        stq.stq_kv_fetch(kv, slots, ko, vo)
        got = [ko, vo]
        for new in (1, 3, 300):
            i = torch.int32
            o = torch.empty(new, 16, d, dtype=q.dtype, device="cuda")
            size = stq.stq_kv_attend_bytes(kv, 1, new, 16, new, L)
            stq.stq_kv_attend(kv, cu(np.arange(3)[None] + first, i), cu([0, new], i), cu([L], i), q[:new], o, d ** -0.5, new, L,
                              work=torch.empty(size, dtype=torch.uint8, device="cuda") if size else None)
            got.append(o)
        torch.cuda.synchronize()
        outs.append(got)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_large_outputs(stq):
    """Outputs larger than the caches take other stores: the same values as calls
    on slices of the tokens, which do not."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    n, heads, kv, d = 4500, 32, 4, 128
    both = torch.randn(n, heads + kv, d, device="cuda", generator=g).bfloat16()
    q, k = both[:, :heads], both[:, heads:]
    table = cu(cos_sin(2048, 64))
    pos = torch.randint(0, 2048, (n,), device="cuda", generator=g).to(torch.int32)
    for dt in (torch.bfloat16, torch.float32):
        whole = [torch.empty(n, heads, d, dtype=dt, device="cuda"), torch.empty(n, kv, d, dtype=dt, device="cuda")]
        parts = [torch.empty_like(x) for x in whole]
        stq.stq_qk_norm_rope(q, k, *whole, pos=pos, cos_sin=table)
        for a in range(0, n, 500):
            s = slice(a, a + 500)
            stq.stq_qk_norm_rope(q[s], k[s], parts[0][s], parts[1][s], pos=pos[s], cos_sin=table)
        assert all(torch.equal(a, b) for a, b in zip(whole, parts))
    cache = stq.make_kv(torch.empty(stq.stq_kv_bytes(300, 64, 8, d), dtype=torch.uint8, device="cuda"), 64, 8, d)
    m = 19000
    kk, vv = (torch.randn(m, 8, d, device="cuda", generator=g).half() for _ in range(2))
    slots = torch.randperm(300 * 64, device="cuda", generator=g)[:m].contiguous()
    stq.stq_kv_store(cache, slots, kk, vv)
    whole, parts = [torch.empty_like(kk) for _ in range(2)], [torch.empty_like(kk) for _ in range(2)]
    stq.stq_kv_fetch(cache, slots, *whole)
    for a in range(0, m, 1000):
        s = slice(a, a + 1000)
        stq.stq_kv_fetch(cache, slots[s], parts[0][s], parts[1][s])
    assert all(torch.equal(a, b) for a, b in zip(whole, parts))


def test_attend_scale_and_large_queries(stq):
    """Negative, zero and large scales; queries far outside binary16's range and
    far below it; rows of zeros."""
    for dtype in ("bf16", "fp16"):
        B = Batch(stq, [100, 37], [1, 3], 4, 2, 64, 32, dtype, seed=3)
        for scale in (-0.2, 0.0, 30.0, 1e-30):
            B.check(B.run(scale=scale))
    B = Batch(stq, [100, 37], [1, 3], 4, 2, 64, 32, "bf16", seed=4)
    for f, s in ((1e30, 1e-31), (1e-30, 1e29), (1e-39, 0.1)):
        q = (B.q.float() * f).to(B.q.dtype)
        q[0, 1] = 0
        B.check(B.run(scale=s, q=q), q=q)


def test_attend_poisoned_tokens(stq):
    """A stored NaN reaches the queries that see it, and no other: positions
    before it, positions whose window has left it, other heads."""
    import torch
    lens, news, window = [90, 70], [30, 1], 12
    for w in (0, window):
        B = Batch(stq, lens, news, 4, 2, 64, 32, "bf16", seed=8)
        slot = np.array([B.table[0, 75 // 32] * 32 + 75 % 32, B.table[1, 1] * 32 + 3])
        k, v = torch.ones(2, 2, 64, device="cuda"), torch.ones(2, 2, 64, device="cuda")
        k[0, 0, 3] = float("nan")
        v[1, 1, 60] = float("inf")
        stq.stq_kv_store(B.kvc, cu(slot.astype(np.int64)), k, v)
        o = B.run(window=w)
        B.check(o, window=w)
        bad = np.isnan(host(o)).all(-1)
        rows = np.arange(60, 90)
        sees = (rows >= 75) & ((rows < 75 + w) if w else True)
        assert np.array_equal(bad[:30, 0], sees) and not bad[:30, 2:].any()


def test_attend_blocks_outside_the_cache(stq):
    """Table entries that name no block hide their tokens (blocks given back
    behind a window), whatever lies in the rest of the table."""
    B = Batch(stq, [300, 170], [1, 50], 4, 2, 128, 32, "bf16", seed=2)
    B.table[0, 2], B.table[0, 5], B.table[1, 0] = -1, 10 ** 6, -2 ** 31
    B.check(B.run())
    B.table[0, :7] = -1
    B.check(B.run(window=60), window=60)


def test_attend_lengths_past_the_table(stq):
    """Lengths beyond the table's columns count as the table's capacity."""
    B = Batch(stq, [64, 64], [1, 2], 4, 2, 64, 32, "bf16", seed=2)
    o = B.run()
    B.lens = np.array([1000, 64])
    p = B.run(max_len=64)
    assert np.array_equal(host(o), host(p))


def test_attend_rows_past_max_new(stq):
    """Query tokens past the stated most are left alone; the others do not change."""
    for cut in (1, 3):
        B = Batch(stq, [100, 50], [5, 2], 4, 1, 128, 32, "bf16", seed=6)
        B.check(B.run(max_new=cut), rows=cut)


def test_attend_strided_rows(stq):
    """q and o as views of wider rows: the rest of the output's rows stays."""
    import torch
    B = Batch(stq, [100, 64], [3, 1], 4, 2, 64, 32, "fp16", seed=6)
    want = B.run()
    wide_q = torch.zeros(B.tok, 7, 64, dtype=torch.float16, device="cuda")
    wide_q[:, 2:6] = B.q
    wide_o = torch.full((B.tok, 6, 64), 5.0, dtype=torch.float16, device="cuda")
    got = B.run(q=wide_q[:, 2:6], o=wide_o[:, 1:5])
    assert torch.equal(got, want) and (wide_o[:, 0] == 5).all() and (wide_o[:, 5] == 5).all()


# --------------------------------------------------- together, graphs, streams

class Layer:
    """One softmax layer of a serving loop, every buffer kept, as a user would hold it."""

    def __init__(self, stq, n, heads, kv, d, T, blocks, cap, dtype="bf16", window=0, sink=0):
        import torch
        i = torch.int32
        z = lambda *s, dtype=i: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.stq, self.n, self.heads, self.kv, self.d, self.T, self.blocks, self.cap = stq, n, heads, kv, d, T, blocks, cap
        self.window, self.sink, self.max_len = window, sink, 400
        self.table = torch.full((n, -(-self.max_len // T)), -1, dtype=i, device="cuda")
        self.free = torch.arange(blocks - 1, -1, -1, dtype=i, device="cuda")
        self.cached, self.new, self.lens, self.start, self.used = z(n), z(n), z(n), z(n + 1), z(1)
        self.pos, self.slots = z(cap), z(cap, dtype=torch.int64)
        self.cs = cu(cos_sin(512, d))
        self.wq, self.wk = torch.linspace(0.5, 1.5, d, device="cuda"), torch.linspace(1.5, 0.5, d, device="cuda")
        self.cache = stq.make_kv(z(stq.stq_kv_bytes(blocks, T, kv, d), dtype=torch.uint8), T, kv, d)
        self.qkv = z(cap, heads + 2 * kv, d, dtype=tt(dtype))
        self.o = z(cap, heads, d, dtype=tt(dtype))
        size = stq.stq_kv_attend_bytes(self.cache, n, cap, heads, cap, self.max_len, window, sink)
        self.work = z(max(size, 16), dtype=torch.uint8)

    def step(self):
        stq, h, kv = self.stq, self.heads, self.kv
        q, k, v = self.qkv[:, :h], self.qkv[:, h:h + kv], self.qkv[:, h + kv:]
        stq.stq_kv_plan(self.cached, self.new, self.free, self.table, self.T, self.blocks, self.start, self.lens, self.pos,
                        self.slots, self.used)
        stq.stq_qk_norm_rope(q, k, q, k, q_weight=self.wq, k_weight=self.wk, pos=self.pos, cos_sin=self.cs)
        stq.stq_kv_store(self.cache, self.slots, k, v)
        stq.stq_kv_attend(self.cache, self.table, self.start, self.lens, q, self.o, self.d ** -0.5, self.cap, self.max_len,
                          self.window, self.sink, self.work)


def test_serving_loop(stq):
    """Prompts, then single tokens, in a padded batch through all four calls:
    every output row against plain binary64 attention over the rotated,
    quantised keys and the quantised values of the whole history."""
    import torch
    for window, sink in ((0, 0), (40, 4)):
        rng = np.random.default_rng(1)
        n, h, kv, d = 3, 4, 2, 64
        Ly = Layer(stq, n, h, kv, d, 32, 40, 128, window=window, sink=sink)
        K, V = [np.zeros((0, kv, d)) for _ in range(n)], [np.zeros((0, kv, d)) for _ in range(n)]
        cached, freed = np.zeros(n, int), 0
        for new in ([70, 5, 31], [1, 1, 1], [1, 0, 2], [3, 90, 1]):
            tok = sum(new)
            raw = rnd(rng, (128, h + 2 * kv, d), "bf16")
            Ly.qkv.copy_(raw)
            Ly.cached.copy_(cu(cached, torch.int32))
            Ly.new.copy_(cu(new, torch.int32))
            Ly.o.fill_(9.0)
            Ly.step()
            torch.cuda.synchronize()
            used = int(Ly.used.item())
            Ly.free = Ly.free[used:].contiguous()
            want = R.plan(cached, new, np.arange(39, -1, -1)[freed:], np.full((n, 13), -1), 32, 40, 128)
            freed += used
            assert want["used"][0] == used and np.array_equal(Ly.start.cpu().numpy(), want["tok_start"])
            assert np.array_equal(Ly.pos.cpu().numpy(), want["pos"])
            x = host(raw)[:tok]
            pos = want["pos"][:tok]
            qr, qs = R.norm_rope(x[:, :h], 1, 1e-6, host(Ly.wq), pos, host(Ly.cs), d, 0)
            kr, ks = R.norm_rope(x[:, h:h + kv], 1, 1e-6, host(Ly.wk), pos, host(Ly.cs), d, 0)
            got = host(Ly.qkv)
            assert (np.abs(got[:tok, :h] - qr) <= R.norm_bound(qr, qs, d, "bf16")).all()
            assert (np.abs(got[:tok, h:h + kv] - kr) <= R.norm_bound(kr, ks, d, "bf16")).all()
            assert np.array_equal(got[tok:], host(raw)[tok:])            # the padding's rows
            for i in range(n):
                s = slice(want["tok_start"][i], want["tok_start"][i + 1])
                if new[i]:
                    K[i] = np.concatenate([K[i], R.value(*R.quantise(got[s, h:h + kv]))])
                    V[i] = np.concatenate([V[i], R.value(*R.quantise(got[s, h + kv:]))])
                for g in range(h):
                    ref, bound = R.attend(got[s, g], K[i][:, g // 2], V[i][:, g // 2], np.ones(len(K[i]), bool), cached[i], d ** -0.5,
                                          window, sink, "bf16")
                    assert (np.abs(host(Ly.o)[s, g] - ref) <= bound).all()
            assert (host(Ly.o)[tok:] == 9).all()
            cached = cached + np.array(new)


def test_l2_norm_feeds_the_state_pool(stq):
    """The L2 form into binary32 is what stq_decode_step takes: the step's
    readout is that of the same step on torch-normalised inputs."""
    import torch
    B, H, d = 4, 2, 128
    desc = stq.make_desc(B, H, d, d, np.array([8, 16], np.int32), np.ones((H, d), np.float32))
    outs = []
    g = torch.Generator(device="cuda").manual_seed(3)
    qk = torch.randn(B, 2 * H, d, device="cuda", generator=g).bfloat16()
    v, S = torch.randn(B, H, d, device="cuda", generator=g), 0.1 * torch.randn(B, H, d, d, device="cuda", generator=g)
    a, b = torch.full((B, H), 0.9, device="cuda"), torch.full((B, H), 0.5, device="cuda")
    q, k = torch.empty(B, H, d, device="cuda"), torch.empty(B, H, d, device="cuda")
    stq.stq_qk_norm_rope(qk[:, :H], qk[:, H:], q, k, norm=stq.STQ_NORM_L2, eps=1e-12)
    f = qk.float()
    f = f / f.square().sum(-1, keepdim=True).sqrt()
    for x, y in ((q, k), (f[:, :H].contiguous(), f[:, H:].contiguous())):
        buf = torch.empty(stq.stq_pool_bytes(desc), dtype=torch.uint8, device="cuda")
        pool = stq.stq_pool_create(desc, buf)
        slots = torch.arange(B, dtype=torch.int32, device="cuda")
        stq.stq_pool_store(pool, slots, S)
        o = torch.empty(B, H, d, device="cuda")
        stq.stq_decode_step(pool, slots, x, y, v, a, b, o)
        torch.cuda.synchronize()
        outs.append(o)
        stq.stq_pool_destroy(pool)
    # inputs a few binary32 steps apart: the readout's binary32 sums over 128 channels differ by that much
    assert (outs[0] - outs[1]).abs().max() <= 128 * 2.0 ** -23 * outs[1].abs().max()


def test_graph_replays(stq):
    """The four calls captured once and replayed over changing buffers, with
    eager work and synchronisations between, give what eager calls give."""
    import torch
    rng = np.random.default_rng(9)
    args = (3, 8, 2, 128, 32, 40, 8)
    A, B = Layer(stq, *args), Layer(stq, *args)
    A.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.step()
    cached, freed = np.zeros(3, int), 0
    for r, new in enumerate(([2, 3, 1], [1, 1, 1], [8, 0, 0], [0, 4, 4], [33 - 30, 1, 1])):
        raw = rnd(rng, (8, 12, 128), "bf16")
        for X in (A, B):
            X.qkv.copy_(raw)
            X.cached.copy_(cu(cached, torch.int32))
            X.new.copy_(cu(new, torch.int32))
            X.o.fill_(1.0)
            X.free.copy_(cu(np.roll(np.arange(40), -freed), torch.int32))
        torch.cuda.synchronize()
        g.replay()
        B.step()
        torch.cuda.synchronize()
        for name in ("o", "table", "lens", "start", "pos", "slots", "used", "qkv"):
            assert torch.equal(getattr(A, name), getattr(B, name)), (r, name)
        freed += int(A.used.item())
        cached = cached + np.array(new)
        torch.ones(1000, device="cuda").sum().item()


def test_two_streams(stq):
    """Two layers on two streams, launched in turn, give what each gives alone."""
    import torch
    rng = np.random.default_rng(4)
    raw = rnd(rng, (64, 12, 128), "bf16")
    want = None
    for pair in (False, True):
        ls = [Layer(stq, 2, 8, 2, 128, 64, 20, 64) for _ in range(2)]
        ss = [torch.cuda.Stream() for _ in range(2)]
        for x in ls:
            x.qkv.copy_(raw)
            x.new.copy_(cu([50, 14], torch.int32))
        torch.cuda.synchronize()
        for x, s in zip(ls, ss if pair else [torch.cuda.current_stream()] * 2):
            with torch.cuda.stream(s):
                x.step()
        torch.cuda.synchronize()
        if want is None:
            want = ls[0].o.clone()
        for x in ls:
            assert torch.equal(x.o, want)


def test_tensor_checks(stq):
    """The compiled checks pass what the calls take and nothing else (the refusals' words are Python's)."""
    import torch
    from quantized_linear_attention_amd import _tensor
    f, i = torch.float32, torch.int32
    t = torch.zeros(5, 6, 64, device="cuda")
    assert _tensor.address(t, f, t.numel(), 0) == t.data_ptr()
    cpu, wide = torch.zeros(5, 6, 64), torch.zeros(5, 10, 64, device="cuda")
    for x, ty, n, dev in ((t, i, t.numel(), 0), (t, f, 7, 0), (t, f, t.numel(), 1), (cpu, f, t.numel(), 0), (cpu, f, t.numel(), -1),
                          (t.transpose(0, 1), f, t.numel(), 0), (None, f, 0, 0), (3, f, 0, 0), (t, "f", t.numel(), 0), (t, f, 2 ** 70, 0),
                          (t, f, None, 0)):
        assert _tensor.address(x, ty, n, dev) is None
    part = wide[:, 2:8]
    assert _tensor.rows(part, 5, 6, 64, 0) == _tensor.rows(part, None, None, None, None) == (part.data_ptr(), 640)
    assert _tensor.rows(t[:1], 1, 6, 64, 0) == (t.data_ptr(), 384)
    assert _tensor.rows(t[0:1].expand(5, 6, 64), 5, 6, 64, 0) == (t.data_ptr(), 0)
    for x, want in ((part, (4, 6, 64, 0)), (part, (5, 5, 64, 0)), (part, (5, 6, 32, 0)), (part, (5, 6, 64, 1)), (part, (5, 6, 64, -1)),
                    (wide[:, ::2], (None,) * 4), (wide[..., ::2], (None,) * 4), (t[0], (None,) * 4), (cpu, (None,) * 4),
                    (None, (None,) * 4), (t, ("5", None, None, None))):
        assert _tensor.rows(x, *want) is None
    q, o = torch.zeros(3, 4, 64, device="cuda").bfloat16(), torch.zeros(3, 4, 64, device="cuda").bfloat16()
    kv = stq.make_kv(torch.zeros(stq.stq_kv_bytes(2, 32, 2, 64), dtype=torch.uint8, device="cuda"), 32, 2, 64)
    ok = dict(table=torch.zeros(1, 2, dtype=i, device="cuda"), tok_start=torch.zeros(2, dtype=i, device="cuda"),
              lens=torch.zeros(1, dtype=i, device="cuda"), q=q, o=o)
    for bad in (dict(table=ok["table"].long()), dict(tok_start=ok["lens"]), dict(lens=ok["lens"].cpu()), dict(q=q.float()), dict(o=o.half()),
                dict(o=o[:2]), dict(q=q.cpu()), dict(q=q[:, :, :32]), dict(q=q[:1].expand(3, 4, 64)), dict(work=torch.zeros(8, device="cuda"))):
        with pytest.raises(stq.StqError):
            stq.stq_kv_attend(kv, **dict(ok, **bad), scale=1.0, max_new=3, max_len=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("news", [1, 7, 12])
def test_attend_of_a_cache_said_to_be_large(stq, dtype, news):
    """Stated lengths whose pages no cache holds: the loads that leave no trace, for one tile of rows, two
    tiles' worth in one, and two tiles."""
    lens = [1, 31, 33, 64, 129, 700, 1555]
    B = Batch(stq, lens, [min(news, n) for n in lens], 8, 2, 128, 32, dtype, seed=news, spare=1)
    for window, sink in ((0, 0), (100, 3)):
        B.check(B.run(window=window, sink=sink, max_len=1 << 20), window, sink)


def test_plan_of_one_buffer(stq):
    """All tensors side by side in one buffer, none reaching into another."""
    import torch
    n, T, cols, tok = 5, 32, 7, 77
    cached, new = [0, 31, 64, 100, 5], [40, 2, 0, 30, 1]
    buf = torch.full((64 + 3 * n + cols * n + 20 + 4 * tok,), -7, dtype=torch.int32, device="cuda")
    at = 0

    def part(m, values=None):
        nonlocal at
        x = buf[at:at + m]
        at += m
        if values is not None:
            x.copy_(cu(np.array(values), torch.int32))
        return x
    used, a, b, f = part(1), part(n, cached), part(n, new), part(20, range(20))
    table, start, lens, pos = part(n * cols).view(n, cols), part(n + 1), part(n), part(tok)
    table.copy_(cu(np.arange(100, 100 + n * cols).reshape(n, cols), torch.int32))
    at += at % 2
    slots = part(2 * tok).view(torch.int64)
    want = R.plan(cached, new, np.arange(20), np.arange(100, 100 + n * cols).reshape(n, cols), T, 200, tok)
    stq.stq_kv_plan(a, b, f, table, T, 200, start, lens, pos, slots, used)
    torch.cuda.synchronize()
    for got, k in ((start, "tok_start"), (lens, "lens"), (pos, "pos"), (slots, "slots"), (table, "table"), (used, "used")):
        assert np.array_equal(got.cpu().numpy(), want[k]), k
    assert a.tolist() == cached and b.tolist() == new and f.tolist() == list(range(20))
    with pytest.raises(stq.StqError):
        stq.stq_kv_plan(a, b, f, table, T, 200, start, a, pos, slots, used)


@pytest.mark.parametrize("news", [[9, 4, 40], [90, 4, 130]])
def test_attend_windows_without_end(stq, news):
    """The largest windows and counts of first tokens are no limit at all, for
    rows at negative positions too."""
    B = Batch(stq, [3, 0, 100], news, 4, 2, 64, 32, "bf16")
    want = B.run()
    B.check(want)
    for window, sink in ((2 ** 31 - 1, 0), (2 ** 31 - 2, 2 ** 31 - 1), (1 << 30, 1), (1, 2 ** 31 - 1)):
        assert np.array_equal(host(B.run(window, sink)), host(want)), (window, sink)


@pytest.mark.parametrize("news,kept", [([3, 6, 2], 5), ([3, 6, 2], 2), ([70, 5, 90], 130), ([4, 300, 7], 150)])
def test_attend_start_offsets_past_the_rows(stq, news, kept):
    """A batch whose offsets go on behind the last row of q (a plan with room for fewer tokens than the
    requests bring): the rows that are there keep their positions."""
    import torch
    B = Batch(stq, [40, 320, 95], news, 4, 2, 64, 32, "bf16")
    whole = B.run()
    B.check(whole)
    for window, sink in ((0, 0), (20, 3)):
        whole = B.run(window, sink)
        o = B.run(window, sink, q=B.q[:kept].clone())
        assert o.shape[0] == kept
        B.check(torch.cat([o, whole[kept:]]), window, sink)


def test_norm_of_more_tokens_than_a_grid_holds(stq):
    """2^26 tokens and a few: as many blocks of 2^20 that all get what one gets alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    m, times, d = 1 << 20, 64, 64
    n = m * times + 5
    one = torch.randn(m, 1, d, device="cuda", generator=g).bfloat16()
    at = torch.randint(0, 300, (m,), device="cuda", generator=g).to(torch.int32)
    table = cu(cos_sin(300, 16))
    want = torch.empty_like(one)
    stq.stq_qk_norm_rope(one, None, want, None, pos=at, cos_sin=table)
    q, pos = torch.empty(n, 1, d, dtype=one.dtype, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    for x, y in ((q, one), (pos, at)):
        x[:m * times].view(times, m, *x.shape[1:]).copy_(y)
        x[m * times:] = y[:5]
    stq.stq_qk_norm_rope(q, None, q, None, pos=pos, cos_sin=table)
    for i in range(times):
        assert torch.equal(q[i * m:(i + 1) * m], want), i
    assert torch.equal(q[m * times:], want[:5])


def test_store_and_fetch_of_more_tokens_than_a_grid_holds(stq):
    """2^29 and a few (token, head) pairs: the tokens that have a slot, some all
    over the call and the last ones, are written and read back, no other."""
    import torch
    heads, d, T = 2048, 64, 32
    n = (1 << 18) + 33
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 130 GiB")
    k, v = (torch.empty(n, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    live = torch.tensor([0, 31, 32, 1 << 16, (1 << 17) - 1, 1 << 17, (1 << 17) + 1, (1 << 18) - 1, 1 << 18, n - 2, n - 1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    a, b = (torch.randn(len(live), heads, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    k[live], v[live] = a, b
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    slots[live] = torch.arange(len(live), device="cuda") + 3
    kv = stq.make_kv(torch.zeros(stq.stq_kv_bytes(1, T, heads, d), dtype=torch.uint8, device="cuda"), T, heads, d)
    few = stq.make_kv(torch.zeros_like(kv.pages), T, heads, d)
    stq.stq_kv_store(few, slots[live], a, b)
    stq.stq_kv_store(kv, slots, k, v)
    assert torch.equal(kv.pages, few.pages)
    want = [torch.empty_like(a) for _ in range(2)]
    stq.stq_kv_fetch(kv, slots[live], *want)
    k[live], v[live] = 7, 7
    k[5], v[n - 9] = 3, 3
    stq.stq_kv_fetch(kv, slots, k, v)
    assert torch.equal(k[live], want[0]) and torch.equal(v[live], want[1])
    assert (k[5] == 3).all() and (v[n - 9] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,d,new,L", [(4, 128, 1, 20011), (3, 64, 8, 20011), (2, 128, 40, 33000), (4, 64, 1, 33000)])
def test_attend_long_requests(stq, dtype, heads, d, new, L):
    """Parts of more than 64 chunks a wave, whose table entries are asked for again, and more than 64 parts of one
    row; blocks outside the cache on both sides of the places where either happens."""
    T = 32
    B = Batch(stq, [L], [new], heads, 1, d, T, dtype, seed=new)
    for at in (3, 63, 64, 65, 255, 256, 257, 320, 511, 512, L // T - 3):
        B.table[0, at] = -1
    i = B.stq
    parts = i.stq_kv_attend_bytes(B.kvc, 1, B.tok, heads, new, L) // (B.tok * heads * (d + 2) * 4)
    assert i.stq_kv_attend_bytes(B.kvc, 1, B.tok, heads, new, 1) == 0
    if L > 30000:
        assert parts > 64
    for hint in (1, L):
        B.check(B.run(max_len=hint))
    B.check(B.run(window=L - 5000, sink=100, max_len=1), L - 5000, 100)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,d,T,longest,new", [(8, 2, 128, 64, 768, 1), (6, 2, 64, 32, 1120, 1), (16, 1, 128, 256, 1021, 1),
                                                      (8, 2, 64, 128, 1100, 4), (3, 3, 128, 32, 900, 5), (64, 16, 128, 64, 2048, 1)])
def test_attend_sixteen_waves(stq, dtype, heads, kv, d, T, longest, new):
    """Requests that one workgroup of sixteen waves takes whole: no workspace; lengths from nothing to the
    longest, windows, a block outside the cache, a token that holds a NaN."""
    import torch
    lens = [longest, 0, 1, 33, 700, 511, longest - 1, 95]
    B = Batch(stq, lens, [min(new, n) for n in lens], heads, kv, d, T, dtype, seed=longest, pad=2)
    assert stq.stq_kv_attend_bytes(B.kvc, len(lens), B.tok, heads, new, longest) == 0
    B.check(B.run())
    B.check(B.run(window=longest - 9, sink=2), longest - 9, 2)
    B.table[4, 1] = -1
    slot = np.array([B.table[0, 600 // T] * T + 600 % T], np.int64)
    k, v = torch.ones(1, kv, d, device="cuda"), torch.ones(1, kv, d, device="cuda")
    k[0, kv - 1, 3] = float("nan")
    stq.stq_kv_store(B.kvc, cu(slot), k, v)
    o = B.run()
    B.check(o)
    g = heads // kv
    assert np.isnan(host(o)[0, -g:]).all() and not np.isnan(host(o)[0, :-g]).any() and not np.isnan(host(o)[B.start[1]:]).any()


@pytest.mark.parametrize("lens,news", [([100, 64, 7], [3, 1, 9]), ([5000, 31], [1, 2]), ([300, 200], [70, 130]), ([5000, 40], [40, 1])])
def test_attend_in_place(stq, lens, news):
    """Output rows in the place of the queries, also as views of one wider buffer; next to them in the
    same rows; any other overlap is refused."""
    import torch
    B = Batch(stq, lens, news, 4, 2, 64, 32, "bf16", seed=len(lens), pad=1)
    want = B.run()
    wide = torch.full((B.tok, 9, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    for first in (1, 5):
        wide[:, 1:5] = B.q
        wide[:, 5:] = 5
        q, o = wide[:, 1:5], wide[:, first:first + 4]
        B.run(q=q, o=o)
        n = int(B.start[-1])
        assert torch.equal(o[:n], want[:n]) and torch.equal(o[n:], B.q[n:] if first == 1 else want[n:])
        assert (wide[:, 0] == 5).all() and (first == 5 or (wide[:, 5:] == 5).all())
    for bad in (wide[:, 2:6], wide[:, :4]):
        with pytest.raises(stq.StqError):
            B.run(q=wide[:, 1:5], o=bad)


def test_attend_parts_of_a_batch(stq):
    """Running requests and prompts in calls of their own on slices of one plan: every row as the reference has
    it, and no row of the other part touched."""
    import torch
    news = [1, 3, 1, 2, 140, 60]
    B = Batch(stq, [700, 33, 1, 95, 140, 333], news, 4, 2, 64, 32, "bf16", seed=3, pad=2)
    i = torch.int32
    table, start, lens = cu(B.table, i), cu(B.start, i), cu(B.lens, i)
    B.check(B.run())
    o = torch.full_like(B.q, 5.0)
    for a, b in ((4, 6), (0, 4)):
        most, longest = int(B.news[a:b].max()), int(B.lens[a:b].max())
        size = stq.stq_kv_attend_bytes(B.kvc, b - a, B.tok, 4, most, longest)
        stq.stq_kv_attend(B.kvc, table[a:b], start[a:b + 1], lens[a:b], B.q, o, B.scale, most, longest,
                          work=torch.empty(size, dtype=torch.uint8, device="cuda") if size else None)
        if a:
            assert (o[:B.start[a]] == 5).all()
    B.check(o)
