"""Attention behind shared prefixes and over lists where their work is cut into many parts: prefixes whose parts are
sized by what all groups have to do, joins of more parts than are asked for at once, more groups and requests than a
wave has lanes for, poisoned and dominant keys in a part, rows of q that are not there."""
import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn import cu, host, rnd, tt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_amd as q
    return q


def i32(x):
    import torch
    return cu(np.asarray(x), torch.int32)


class Shared:
    """Requests behind shared prefixes: `before` in no group, then groups of sizes[g] behind prefix[g] tokens, then
    `behind` in no group; own[i] tokens of each one's own, the last new[i] of them queries.  A prefix is stored once."""

    def __init__(self, stq, sizes, prefix, own, new, heads, kv, d, T, dtype, seed, before=0, behind=0, keys=None, values=None):
        rng = np.random.default_rng(seed)
        self.stq, self.heads, self.kv, self.d, self.T, self.dtype = stq, heads, kv, d, T, dtype
        self.groups = before + np.concatenate([[0], np.cumsum(sizes)])
        self.prefix = np.array(prefix)
        n = before + sum(sizes) + behind
        self.own, self.new = np.broadcast_to(own, n).astype(int), np.broadcast_to(new, n).astype(int)
        head = np.zeros(n, int)
        for g, p in enumerate(prefix):
            head[self.groups[g]:self.groups[g + 1]] = p
        self.lens = head + self.own
        nb = sum(p // T for p in prefix) + int((-(-self.own // T)).sum()) + 3
        ids, at = rng.permutation(nb), 0
        self.table = np.full((n, int((-(-self.lens // T)).max()) + 1), -1)
        slots = []
        for g, p in enumerate(prefix):
            self.table[self.groups[g]:self.groups[g + 1], :p // T] = ids[at:at + p // T]
            slots.append((ids[at:at + p // T, None] * T + np.arange(T)).ravel())
            at += p // T
        for i in range(n):
            m = -(-self.own[i] // T)
            self.table[i, head[i] // T:head[i] // T + m] = ids[at:at + m]
            slots.append((ids[at:at + m, None] * T + np.arange(T)).ravel()[:self.own[i]])
            at += m
        slots = np.concatenate(slots)
        import torch
        self.pages = torch.full((stq.stq_kv_bytes(nb, T, kv, d),), 0xFF, dtype=torch.uint8, device="cuda")
        self.kvc = stq.make_kv(self.pages, T, kv, d)
        shape = (len(slots), kv, d)
        k = rng.standard_normal(shape) if keys is None else keys(rng, shape)
        # (a mean of its own in every 256 tokens: a part that is lost or counted twice moves the output)
        v = rng.standard_normal(shape) + 2 * np.repeat(rng.standard_normal((len(slots) // 256 + 1, kv, d)), 256, 0)[:len(slots)] \
            if values is None else values(rng, shape)
        stq.stq_kv_store(self.kvc, cu(slots), cu(k, tt("fp32")), cu(v, tt("fp32")))
        self.start = np.concatenate([[0], np.cumsum(self.new)])
        self.q = rnd(rng, (int(self.start[-1]) + 2, heads, d), dtype)

    def write(self, i, s, k, v):
        """Key and value [kv][d] of position s of request i."""
        slot = self.table[i, s // self.T] * self.T + s % self.T
        self.stq.stq_kv_store(self.kvc, cu([slot]), cu(np.asarray(k)[None], tt("fp32")), cu(np.asarray(v)[None], tt("fp32")))

    def run(self, q=None, o=None, max_own=None, max_prefix=None, fill=0xFF, scale=None):
        import torch
        stq, n = self.stq, len(self.lens)
        q = self.q if q is None else q
        o = torch.full_like(q, 5.0) if o is None else o
        self.scale = self.d ** -0.5 if scale is None else scale
        m, w, p = int(self.new.max()), int(self.own.max()) if max_own is None else max_own, int(max(self.prefix)) if max_prefix is None else max_prefix
        size = stq.stq_kv_attend_shared_bytes(self.kvc, n, q.shape[0], self.heads, len(self.prefix), m, w, p)
        work = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        stq.stq_kv_attend_shared(self.kvc, i32(self.table), i32(self.start), i32(self.lens), i32(self.groups), i32(self.prefix), q, o,
                                 self.scale, m, w, p, work)
        torch.cuda.synchronize()
        return o

    def cached(self):
        """Keys and values of all blocks, [block][T][kv][d] in binary64; NaN where poisoned or unwritten."""
        c = R.Cache(self.kvc.desc.n_blocks, self.T, self.kv, self.d)
        kc, vc, ks, vs = c.parts(self.pages.cpu().numpy())
        out = []
        for code, sc in ((kc, ks), (vc, vs)):
            x = np.stack([code & 15, code >> 4], -1).reshape(code.shape[:-1] + (self.d,))
            e = sc.astype(np.int64).swapaxes(-1, -2)
            y = R.value(x, np.where(e == 255, 0, e - 127))
            out.append(np.where(np.repeat(e == 255, 32, -1), np.nan, y).transpose(0, 2, 1, 3))
        return out

    def check(self, o, rows=None):
        """Every row against binary64, with the bound of attn_ref.attend, in which |v - o| is taken as at most |v| + |o|."""
        K, V = self.cached()
        o, q = host(o), host(self.q)
        g, scale = self.heads // self.kv, float(np.float32(self.scale))
        end = len(o) if rows is None else rows
        for i, (L, m) in enumerate(zip(self.lens, self.new)):
            t0, t1 = self.start[i], min(self.start[i + 1], end)
            if t1 <= t0:
                continue
            blk = self.table[i, :-(-L // self.T)]
            k, v = (x[blk].reshape(-1, self.kv, self.d)[:L] for x in (K, V))
            p = np.repeat(L - m + np.arange(t1 - t0), g)
            see = np.arange(L) <= p[:, None]                                    # [rows][L]
            for h in range(self.kv):
                x = q[t0:t1, h * g:(h + 1) * g].reshape(-1, self.d)
                nan = (see & np.isnan(k[:, h]).any(1)).any(1)
                kk, vv = np.nan_to_num(k[:, h]), np.nan_to_num(v[:, h])
                logit = np.where(see, scale * (x @ kk.T), -np.inf)
                size = np.where(see, abs(scale) * (np.abs(x) @ np.abs(kk).T), 0)
                w = np.exp(logit - logit.max(1, keepdims=True))
                tot = w.sum(1, keepdims=True)
                want = (w @ vv) / tot
                big = np.where(see, np.abs(logit), 0)
                err = self.d * 2.0 ** -23 * (size + size.max(1, keepdims=True)) + 4 * 2.0 ** -24 * (big + big.max(1, keepdims=True)) + 2.0 ** -21 + 2.0 ** -10
                err = np.where(see, err * w + 2.0 ** -24, 0)
                steps = (L / 32 + 40) * 2.0 ** -23
                bound = ((err + steps * w) @ np.abs(vv) + (err.sum(1, keepdims=True) + steps * tot) * np.abs(want)) / tot
                bound += R.HALF[self.dtype] * np.abs(want) * 1.001 + 2.0 ** -25
                got = o[t0:t1, h * g:(h + 1) * g].reshape(-1, self.d)
                assert np.isnan(got[nan]).all() and not np.isnan(got[~nan]).any(), (i, h)
                off = np.abs(got - want)[~nan]
                assert (off <= bound[~nan]).all(), (i, h, (off / bound[~nan]).max())
        assert (o[min(self.start[-1], end):] == 5).all()


def ragged(seed, n, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi + 1, n)


# Workgroups of a prefix' parts are to fill the card once: 512 over the heads, 64 of them for eight.  With parts of the
# least size these would be more (tiles of 16 rows, or of 128 from 64 rows a group on, times parts), so that parts grow.
@pytest.mark.parametrize("heads,d,sizes,prefix,new", [
    (16, 64, [20] * 8, [2048, 2048, 1920, 2048, 1024, 2048, 2016, 2048], 1),    # few rows: 24 tiles, 3 parts
    (32, 64, [60, 58, 60, 59], [2048, 2048, 2048, 2240], 2),                    # tiles of 128 rows, few own rows: 16 tiles, 4 and 5 parts
    (32, 128, [20, 20, 19], [2048, 2080, 2048], 6),                             # 24 own rows: 12 tiles, 6 parts
    (32, 64, [6, 5], [2048, 2304], 33),                                         # prompts on both sides
])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_parts_of_prefixes_grow(stq, dtype, heads, d, sizes, prefix, new):
    n = sum(sizes) + 3
    x = Shared(stq, sizes, prefix, new + ragged(1, n, 0, 60), new, heads, 8, d, 32, dtype, seed=new, before=1, behind=2)
    x.check(x.run())
    x.check(x.run(max_own=100000, max_prefix=1))


@pytest.mark.parametrize("kv,heads", [(2, 4), (8, 8)])
def test_parts_of_many_groups(stq, kv, heads):
    """More groups than a wave has lanes: prefixes of several parts, of which there is room for all (two heads), or
    for one a group (eight)."""
    rng = np.random.default_rng(3)
    sizes = [int(rng.integers(1, 3)) if g % 9 else 0 for g in range(75)]
    prefix = [32 * int(rng.integers(20, 33)) for _ in sizes]
    prefix[70] = 4096
    n = sum(sizes) + 2
    x = Shared(stq, sizes, prefix, 1 + ragged(2, n, 0, 50), 1, heads, kv, 64, 32, "bf16", seed=kv, before=2)
    x.check(x.run())


@pytest.mark.parametrize("new", [1, 5])
def test_parts_of_many_requests(stq, new):
    """More requests than a wave keeps: 325 behind five prefixes in parts that grow."""
    x = Shared(stq, [65] * 5, [4096, 3200, 4096, 2048, 1600], new + ragged(4, 325, 0, 40), new, 32, 8, 64, 64, "bf16", seed=new)
    x.check(x.run())


# (members, heads over one, prefix, own tokens): parts of the prefix and of the own tokens that a row joins.  Eight are
# asked for at once, then 24 more at a time; past 64 a lane holds two of their statistics.
@pytest.mark.parametrize("members,heads,prefix,own", [
    (3, 4, 8192, 6000),          # 16 and 12
    (3, 4, 2048, 16000),         # 6 and 32
    (2, 2, 32768, 16000),        # 64 and 32
    (5, 16, 8192, 6000),         # the prefix by tiles of 128 rows
    (4, 20, 8192, 6000),         # rows of 32
])
def test_joins_of_many_parts(stq, members, heads, prefix, own):
    x = Shared(stq, [members], [prefix], own - 7 * np.arange(members), 1, heads, 1, 64, 64, "bf16", seed=heads)
    x.check(x.run())
    x.check(x.run(max_own=64))


@pytest.mark.parametrize("heads,sizes,prefix,new", [(4, [3, 2], [512, 1024], 1), (16, [30, 2], [512, 1024], 2), (8, [3, 3], [1024, 320], 40)])
def test_poisoned_keys(stq, heads, sizes, prefix, new):
    """A poisoned key of a shared prefix reaches every row behind it through its head, one of a request's own the rows
    at and past it, and nothing else."""
    x = Shared(stq, sizes, prefix, new + 45, new, heads, 2, 64, 32, "bf16", seed=new, before=1)
    first = x.groups[0]
    bad = np.zeros((2, 64))
    bad[1, 3] = np.inf
    x.write(first, 300, bad, np.zeros((2, 64)))              # of the first group's prefix, head 1
    bad = bad[::-1].copy()
    last = len(x.lens) - 1
    x.write(last, x.lens[last] - new, bad, np.zeros((2, 64)))      # the last request's first new token, head 0
    o = x.run()
    x.check(o)
    nan, g = np.isnan(host(o)).any(-1), heads // 2
    s, e = x.start[first], x.start[x.groups[1]]
    assert nan[s:e, g:].all() and not nan[s:e, :g].any() and not nan[:s].any()
    assert nan[x.start[last]:x.start[last + 1], :g].all() and not nan[e:x.start[last]].any() and not nan[e:, g:].any()


STEEP = [("bf16", 100.0, 13, 0.088), ("bf16", 2.0 ** 100, 0, -0.088), ("bf16", 2.0 ** 127, 13, 8.0), ("bf16", 2.0 ** -100, -23, 3e38),
         ("fp16", 6e4, 13, 30.0), ("fp16", 6e4, 13, -3e38)]


def steep_keys(sign, exp):
    def make(rng, shape):
        K = rng.choice([0.0, 0.5, 1.0, 1.5, 2.0], shape) * sign * np.where(rng.random(shape) < 0.3, -1, 1)
        return K * 2.0 ** exp
    return make


@pytest.mark.parametrize("dtype,mag,exp,scale", STEEP)
@pytest.mark.parametrize("heads,members,new,d,own", [(2, 3, 1, 64, 300), (4, 3, 1, 128, 2000), (8, 12, 2, 64, 500), (8, 3, 20, 128, 700)])
def test_steep_rows(stq, dtype, mag, exp, scale, heads, members, new, d, own):
    """Logits of any finite size through parts of two kernels.  Tokens with the same largest logit lie in two parts of
    the prefix and in a request's own part, all others far below: the output is the mean of their values (products, sums
    and the mean of one, two or four are exact; two binary32 steps for the quotient and the product with it, then the
    output's own rounding)."""
    import torch
    rng = np.random.default_rng(d + new)
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    x = Shared(stq, [members], [1024], own, new, heads, 1, d, 32, dtype, seed=d, keys=steep_keys(sign, exp),
               values=lambda r, s: r.standard_normal(s))
    top, zero = 4 * sign * 2.0 ** exp, rng.standard_normal((4, 1, d))
    x.write(0, 37, top[None], zero[0])                      # in the prefix: its first part and its last
    x.write(0, 1000, top[None], zero[1])
    for s in (1024 + 5, 1024 + own - new - 3):              # of request 1's own: the first part and the last
        x.write(1, s, top[None], zero[2 + (s > 1024 + 5)])
    x.write(0, 700, -1.5 * top[None], zero[0])              # and the most negative product, for queries that turn
    V = x.cached()[1]
    at = lambda i, s: V[x.table[i, s // 32], s % 32, 0]  # noqa: E731
    for flip in (1.0, -1.0):
        q = torch.as_tensor(np.broadcast_to(sign * mag * np.sign(scale) * flip, (x.q.shape[0], heads, d)).copy(), device="cuda").to(tt(dtype))
        for kw in ({}, dict(max_own=100000, max_prefix=100000), dict(max_own=1, max_prefix=1)):
            o = host(x.run(q=q, scale=scale, **kw))
            for i in range(members):
                tops = [(i, 700)] if flip < 0 else [(i, 37), (i, 1000)] + ([(1, 1029), (1, 1024 + own - new - 3)] if i == 1 else [])
                want = np.mean([at(*t) for t in tops], 0)
                got = o[x.start[i]:x.start[i + 1]]
                assert np.isfinite(got).all()
                assert (np.abs(got - want) <= (R.HALF[dtype] + 2.0 ** -21) * np.abs(want) + 2.0 ** -25).all(), (flip, kw, i, np.abs(got - want).max())


@pytest.mark.parametrize("dtype,mag,exp,scale", STEEP)
@pytest.mark.parametrize("heads,kv,n_sel,many", [(4, 1, 60, False), (4, 1, 14, False), (20, 1, 40, False), (4, 1, 9, True)])
def test_steep_lists(stq, dtype, mag, exp, scale, heads, kv, n_sel, many):
    """The same over lists: in parts with a join, by sixteen waves, in rows of 32, by one wave a list."""
    import torch
    d, T, L = 128, 64, 64 * 64
    rng = np.random.default_rng(n_sel)
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    new = 2100 if many else 1
    x = Shared(stq, [], [], L, new, heads, kv, d, T, dtype, seed=n_sel, behind=1, keys=steep_keys(sign, exp), values=lambda r, s: r.standard_normal(s))
    top, v = 4 * sign * 2.0 ** exp, rng.standard_normal((3, 1, d))
    x.write(0, 70, top[None], v[0])                          # blocks 1 and 20; block 11 the most negative product
    x.write(0, 20 * T + 9, top[None], v[1])
    x.write(0, 11 * T + 3, -1.5 * top[None], v[2])
    cols = np.sort(np.concatenate([[1, 11, 20], rng.permutation(np.r_[0, 2:11, 12:20, 21:30 if many else 64])[:n_sel - 3]]))
    tok = x.q.shape[0]
    sel = i32(np.broadcast_to(cols, (tok, kv, n_sel)).copy())
    V = x.cached()[1]
    at = lambda s: V[x.table[0, s // T], s % T, 0]  # noqa: E731
    size = stq.stq_kv_attend_blocks_bytes(x.kvc, 1, tok, heads, n_sel, new)
    work = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
    for flip in (1.0, -1.0):
        q = torch.as_tensor(np.broadcast_to(sign * mag * np.sign(scale) * flip, (tok, heads, d)).copy(), device="cuda").to(tt(dtype))
        o = torch.full_like(q, 5.0)
        stq.stq_kv_attend_blocks(x.kvc, i32(x.table), i32(x.start), i32(x.lens), sel, q, o, scale, new, work)
        want = np.mean([at(70), at(20 * T + 9)], 0) if flip > 0 else at(11 * T + 3)
        got = host(o)[:new]
        assert (np.abs(got - want) <= (R.HALF[dtype] + 2.0 ** -21) * np.abs(want) + 2.0 ** -25).all(), (flip, np.abs(got - want).max())


def test_the_same_call_gives_the_same_bits(stq):
    """Whatever the workspace holds, and again and again: no result goes by the order of workgroups."""
    import torch
    for heads, sizes, prefix, new in ((32, [32, 28], [2048, 1088], 1), (8, [8], [1024], 1), (32, [5, 6], [640, 1024], 40)):
        x = Shared(stq, sizes, prefix, new + ragged(5, sum(sizes), 0, 900), new, heads, 8, 128, 64, "bf16", seed=heads)
        o = x.run()
        for fill in (0, 0x3F, 0xFF, 0xFF):
            assert torch.equal(x.run(fill=fill), o)
        cols = x.table.shape[1]
        rng = np.random.default_rng(1)
        sel = i32(np.sort(np.stack([rng.permutation(cols)[:12] for _ in range(x.q.shape[0] * 8)]).reshape(-1, 8, 12), -1))
        outs = []
        for fill in (0, 0xFF, 0xFF):
            size = stq.stq_kv_attend_blocks_bytes(x.kvc, len(x.lens), x.q.shape[0], heads, 12, new)
            work = torch.full((size,), fill, dtype=torch.uint8, device="cuda") if size else None
            outs.append(torch.full_like(x.q, 5.0))
            stq.stq_kv_attend_blocks(x.kvc, i32(x.table), i32(x.start), i32(x.lens), sel, x.q, outs[-1], x.scale, new, work)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[1], outs[2])


@pytest.mark.parametrize("heads,sizes,new", [(4, [3, 3], 3), (32, [9, 9], 2), (8, [3, 2], 40)])
def test_rows_of_q_that_are_not_there(stq, heads, sizes, new):
    """Fewer rows of q than new tokens: the others' positions stay, and the prefix is cut by all of them."""
    n = sum(sizes) + 2
    x = Shared(stq, sizes, [512, 256], new + ragged(7, n, 0, 70), new, heads, 2, 64, 32, "bf16", seed=heads, before=1, behind=1)
    for rows in (1, new + 1, int(x.start[-3]) + 1, int(x.start[-2]) - 1):
        x.check(x.run(q=x.q[:rows].clone()), rows=rows)
