"""Host checks of the entry points for long contexts (no GPU): sizes, and every refusal before anything is enqueued."""
import ctypes

import pytest

from test_attn_abi import D, P, Fake, ad, kvd


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_amd as q
    return q


@pytest.fixture(scope="module")
def L(stq):
    from quantized_linear_attention_amd import _lib
    return _lib._L


def sd(**kw):
    from quantized_linear_attention_amd._lib import _SelectDesc
    d = dict(n_req=3, n_tok=5, n_kv_heads=2, block_tokens=64, table_cols=40, n_sel=8, n_first=1, n_last=2, max_new=2)
    d.update(kw)
    return _SelectDesc(*[d[f[0]] for f in _SelectDesc._fields_])


def gd(n_groups=2, max_prefix=128):
    from quantized_linear_attention_amd._lib import _SharedDesc
    return _SharedDesc(n_groups, max_prefix)


ref = ctypes.byref
FULL = 10 * 2 * 64 * 136                                 # bytes of kvd()'s cache
FAR = P(1 << 40)                                         # far from D and everything that starts there


def test_bounds_size_and_refusals(L):
    assert L.stq_kv_bounds_bytes(ref(kvd())) == 10 * 2 * 2 * 128
    assert L.stq_kv_bounds_bytes(ref(kvd(n_blocks=2 ** 31 - 1, n_kv_heads=8))) == (2 ** 31 - 1) * 8 * 256
    assert L.stq_kv_bounds_bytes(ref(kvd(d=96))) == 0

    def call(d=None, cache=D, size=FULL, n=3, max_new=2, table=D, cols=5, tok=D, len=D, bounds=FAR):
        return L.stq_kv_bounds(ref(d or kvd()), cache, size, n, max_new, table, cols, tok, len, bounds, None)
    for kw in (dict(d=kvd(d=32)), dict(n=-1), dict(max_new=0), dict(cols=0), dict(cols=1 << 25), dict(table=None), dict(tok=None),
               dict(len=None), dict(bounds=None), dict(bounds=D), dict(bounds=P(0x10000 + FULL - 16)), dict(bounds=P(0x10000 - 5104))):
        assert call(**kw) == -1, kw
    for kw in (dict(cache=None), dict(cache=P(0x10008)), dict(size=FULL - 1), dict(bounds=P((1 << 40) + 8))):
        assert call(**kw) == -2, kw
    assert call(n=0, table=None) == 0
    # a launch of 2^32 threads: more (request, block) pairs than it takes
    assert call(n=1 << 23, max_new=1) == -5 and call(n=1 << 12, max_new=1 << 18, cols=1 << 13) == -5


def test_score_refusals(L):
    def call(a=None, d=None, bounds=FAR, table=D, tok=D, len=D, q=D, score=P(1 << 41)):
        return L.stq_kv_score(ref(d or kvd()), ref(a or ad()), bounds, table, tok, len, q, score, None)
    for kw in (dict(n_req=-1), dict(n_tok=-1), dict(n_heads=3), dict(type=2), dict(table_cols=0), dict(max_new=0), dict(max_len=0),
               dict(window=1), dict(n_sink=1), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(ad(**kw)) == -1, kw
    assert call(d=kvd(d=96)) == -1
    for name in ("bounds", "table", "tok", "len", "q", "score"):
        assert call(**{name: None}) == -1, name
    # score over the bounds or over the queries (3 rows of 512 elements of 2 bytes; score: 3 * 2 * 5 floats)
    for at in (1 << 40, (1 << 40) + 5120 - 16, (1 << 40) - 112, 0x10000, 0x10000 + 3 * 1024 - 16, 0x10000 - 112):
        assert call(score=P(at)) == -1, at
    for kw in (dict(q=P(0x10008)), dict(bounds=P((1 << 40) + 4)), dict(score=P((1 << 41) + 8)), dict(a=ad(q_stride=504)), dict(a=ad(q_stride=516))):
        assert call(**kw) == -2, kw
    assert call(ad(n_req=0), q=None) == 0 and call(ad(n_tok=0), q=None) == 0
    assert call(ad(n_req=1 << 23)) == -5
    assert call(ad(n_req=1, max_new=1 << 26)) == -5


@pytest.mark.parametrize("a,d", [(dict(n_req=1 << 23), {}), (dict(n_req=(1 << 24) // 3 + 1), dict(n_kv_heads=3)), (dict(max_new=4194241, n_heads=6), {}),
                                 (dict(max_new=8388481, n_heads=4), {}), (dict(max_new=16776961, n_heads=2), {})])
def test_score_just_past_its_limits(L, a, d):
    """The first number of (request, head) pairs and of new tokens (six, four and two heads over two) that is refused."""
    a = dict(dict(n_heads=d.get("n_kv_heads", 2), q_stride=6 * 128), **a)
    assert L.stq_kv_score(ref(kvd(**d)), ref(ad(**a)), FAR, D, D, D, D, P(1 << 41), None) == -5


def test_select_refusals(L):
    def call(c=None, tok=D, len=D, score=D, sel=FAR):
        return L.stq_kv_select(ref(c or sd()), tok, len, score, sel, None)
    for kw in (dict(n_req=-1), dict(n_tok=-1), dict(n_tok=(1 << 28) + 1), dict(n_kv_heads=0), dict(n_kv_heads=4097), dict(block_tokens=48),
               dict(table_cols=0), dict(table_cols=1 << 25), dict(max_new=0), dict(n_sel=0), dict(n_first=-1), dict(n_last=-1),
               dict(n_first=7, n_last=2), dict(n_first=2 ** 31 - 1, n_last=2 ** 31 - 1)):
        assert call(sd(**kw)) == -1, kw
    assert L.stq_kv_select(None, D, D, D, FAR, None) == -1
    for name in ("tok", "len", "score", "sel"):
        assert call(**{name: None}) == -1, name
    for at in (0x10000, 0x10000 + 5 * 2 * 40 * 4 - 16, 0x10000 - 5 * 2 * 8 * 4 + 16):
        assert call(sel=P(at)) == -1, at
    assert call(score=P(0x10008)) == -2 and call(sel=P((1 << 40) + 4)) == -2
    assert call(sd(n_req=0), sel=None) == 0 and call(sd(n_tok=0), sel=None) == 0
    assert call(sd(table_cols=32769)) == -5
    assert call(sd(n_req=1 << 20, max_new=1 << 12)) == -5
    assert call(sd(n_req=1 << 20, max_new=4, table_cols=4096)) == -5         # 1,024 threads a row
    # the first number of rows that is refused: 64 threads a row to 2,048 columns (four rows a workgroup), 1,024 past that
    for cols in (1, 512, 513, 2048):
        assert call(sd(n_req=67108861, max_new=1, n_kv_heads=1, table_cols=cols)) == -5, cols
    for cols in (2049, 32768):
        assert call(sd(n_req=4194304, max_new=1, n_kv_heads=1, table_cols=cols)) == -5, cols


def test_blocks_refusals(L):
    def call(a=None, k=4, d=None, cache=D, size=FULL, work=P(1 << 43), wbytes=1 << 40, **at):
        p = dict(table=D, tok=D, len=D, sel=FAR, q=D, o=P(0x20000))
        p.update(at)
        return L.stq_kv_attend_blocks(ref(d or kvd()), cache, size, ref(a or ad()), k, p["table"], p["tok"], p["len"], p["sel"], p["q"],
                                      p["o"], work, wbytes, None)
    for kw in (dict(n_req=-1), dict(n_tok=-1), dict(n_heads=3), dict(type=2), dict(table_cols=0), dict(max_new=0), dict(max_len=0),
               dict(window=1), dict(n_sink=1), dict(scale=float("nan"))):
        assert call(ad(**kw)) == -1, kw
    for k in (0, -1, (1 << 24) + 1):
        assert call(k=k) == -1, k
    for name in ("table", "tok", "len", "sel", "q", "o"):
        assert call(**{name: None}) == -1, name
    for o in (0x10000 + 16, 0x10000 - 16, 1 << 40, (1 << 40) + 3 * 2 * 4 * 4 - 16):
        assert call(o=P(o)) == -1, o
    for kw in (dict(cache=P(0x10008)), dict(size=FULL - 1), dict(q=P(0x10008)), dict(o=P(0x20002)), dict(sel=P((1 << 40) + 4)),
               dict(a=ad(q_stride=504)), dict(a=ad(o_stride=516))):
        assert call(**kw) == -2, kw
    # lists whose work is split take a workspace of the stated size
    need = L.stq_kv_attend_blocks_bytes(ref(kvd()), ref(ad()), 100)
    assert need > 0 and L.stq_kv_attend_blocks_bytes(ref(kvd()), ref(ad()), 1) == 0
    assert call(k=100, work=None) == -2 and call(k=100, wbytes=need - 1) == -2 and call(k=100, work=P(0x10004)) == -2
    assert L.stq_kv_attend_blocks_bytes(ref(kvd()), ref(ad(window=3)), 100) == 0
    assert call(ad(n_req=0)) == 0 and call(ad(n_tok=0)) == 0
    assert call(ad(n_req=1 << 20, max_new=1 << 12)) == -5


def test_shared_refusals(L):
    def call(a=None, g=None, d=None, cache=D, size=FULL, work=P(1 << 43), wbytes=1 << 42, **at):
        p = dict(table=D, tok=D, len=D, group=D, prefix=D, q=D, o=P(0x20000))
        p.update(at)
        g = g or gd()
        return L.stq_kv_attend_shared(ref(d or kvd()), cache, size, ref(a or ad()), ref(g), p["table"], p["tok"], p["len"], p["group"],
                                      p["prefix"], p["q"], p["o"], work, wbytes, None)
    for kw in (dict(n_req=-1), dict(n_tok=-1), dict(n_heads=3), dict(type=2), dict(table_cols=0), dict(max_new=0), dict(max_len=0),
               dict(window=1), dict(n_sink=1), dict(scale=float("inf"))):
        assert call(ad(**kw)) == -1, kw
    assert call(g=gd(-1)) == -1 and call(g=gd(2, -1)) == -1
    for name in ("table", "tok", "len", "group", "prefix", "q", "o"):
        assert call(**{name: None}) == -1, name
    for o in (0x10000 + 16, 0x10000 - 16):
        assert call(o=P(o)) == -1, o
    for kw in (dict(cache=None), dict(size=FULL - 1), dict(q=P(0x10008)), dict(o=P(0x20002)), dict(a=ad(q_stride=504)), dict(a=ad(o_stride=516))):
        assert call(**kw) == -2, kw
    need = L.stq_kv_attend_shared_bytes(ref(kvd()), ref(ad()), ref(gd()))
    assert need > 0 and call(work=None) == -2 and call(wbytes=need - 1) == -2 and call(work=P(0x10004)) == -2
    for g in (gd(0, 0), gd(1, 0), gd(1, 2 ** 31 - 1), gd(2 ** 20, 64)):      # a size for every description
        assert L.stq_kv_attend_shared_bytes(ref(kvd()), ref(ad(max_len=2 ** 30)), ref(g)) > 0
    assert L.stq_kv_attend_shared_bytes(ref(kvd()), ref(ad()), ref(gd(-1))) == 0
    assert call(ad(n_req=0)) == 0 and call(ad(n_tok=0)) == 0
    assert call(ad(n_req=1 << 20, max_new=1 << 12)) == -5
    assert call(g=gd(1 << 24)) == -5                                         # a launch takes a workgroup and more a group


@pytest.mark.parametrize("n_req,n_kv_heads", [(1, 8), (4, 8), (16, 8), (30, 8), (32, 8), (64, 4), (200, 1)])
def test_own_tokens_are_split_among_the_waves_there_are(L, n_req, n_kv_heads):
    """Requests' own tokens behind shared prefixes: one part for every 12 chunks of 32 tokens, until there are 512
    workgroups, at every length.  (Each is taken by four waves; a part that only sixteen would be enough for is none.)
    The workspace tells: of n rows of a head's d outputs and 2 statistics, one a part, and one part of the prefix."""
    d, heads = 128, 4 * n_kv_heads
    g = gd(n_groups=0, max_prefix=0)
    for own in range(32, 2500, 32):
        chunks = own // 32
        kv = kvd(n_kv_heads=n_kv_heads)
        a = ad(n_req=n_req, n_tok=n_req, n_heads=heads, max_len=own, q_stride=heads * d, o_stride=heads * d)
        parts, rest = divmod(L.stq_kv_attend_shared_bytes(ref(kv), ref(a), ref(g)) - (n_req * 4 + 19) // 16 * 16, n_req * heads * (d + 2) * 4)
        most = max(1, min(512 // (n_req * n_kv_heads), chunks // 12))
        per = (-(-chunks // most) + 3) // 4 * 4                 # whole chunks for each wave
        assert rest == 0 and parts - 1 == -(-chunks // per), (own, parts, most)


def test_lists_of_many_pairs_are_whole(L):
    """From 2,048 (token, head) pairs on no list is split, however long: a wave on its own writes no parts."""
    for n_req, max_new, hkv in ((256, 1, 8), (1, 2048, 1), (683, 3, 1), (64, 16, 2), (5000, 1, 8)):
        kv, a = kvd(n_kv_heads=hkv), ad(n_req=n_req, n_tok=n_req * max_new, n_heads=2 * hkv, max_new=max_new)
        for n_sel in (1, 2, 100, 32768, 1 << 24):
            assert L.stq_kv_attend_blocks_bytes(ref(kv), ref(a), n_sel) == 0, (n_req, n_sel)


def test_binding_refusals(stq, monkeypatch):
    """Shapes, types, devices and values that the binding does not pass on."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # some refusals are the library's own
    b, f, i, u, e = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e5m2
    E = stq.StqError
    kv = stq.make_kv(Fake([FULL], u), 64, 2, 128)
    assert stq.stq_kv_bounds_bytes(kv) == 10 * 2 * 2 * 128
    table, start, lens = Fake([3, 5], i), Fake([4], i), Fake([3], i)
    bounds, q, o = Fake([10, 2, 2, 128], e, ptr=1 << 40), Fake([6, 4, 128], b), Fake([6, 4, 128], b, ptr=0x20000)
    score, sel = Fake([6, 2, 5], f, ptr=1 << 41), Fake([6, 2, 3], i, ptr=1 << 42)
    big = Fake([1 << 20], u, ptr=1 << 43)
    calls = [
        (stq.stq_kv_bounds, dict(kv=kv, table=table, tok_start=start, lens=lens, bounds=bounds, max_new=2),
         [dict(bounds=Fake([10, 2, 2, 128], u)), dict(bounds=Fake([9, 2, 2, 128], e)), dict(table=Fake([15], i)), dict(tok_start=Fake([3], i)),
          dict(lens=Fake([3], torch.int64)), dict(lens=Fake([3], i, "cuda:1")), dict(max_new=1.5), dict(max_new=2 ** 31), dict(max_new=0)]),
        (stq.stq_kv_score, dict(kv=kv, bounds=bounds, table=table, tok_start=start, lens=lens, q=q, score=score, scale=0.1, max_new=2, max_len=300),
         [dict(score=Fake([6, 2, 4], f)), dict(score=Fake([6, 2, 5], b)), dict(q=Fake([6, 4, 64], b)), dict(q=Fake([6, 4, 128], f)),
          dict(q=Fake([6, 4, 128], b, stride=(1024, 256, 1))), dict(q=Fake([6, 3, 128], b)), dict(max_len=2 ** 31), dict(scale="1"),
          dict(scale=1e39), dict(table=Fake([3, 5], i, "cuda:1")), dict(score=Fake([6, 2, 5], f, ptr=0x10000))]),
        (stq.stq_kv_select, dict(score=score, tok_start=start, lens=lens, sel=sel, block_tokens=64, max_new=2),
         [dict(sel=Fake([6, 1, 3], i)), dict(sel=Fake([5, 2, 3], i)), dict(sel=Fake([6, 2, 3], torch.int64)), dict(score=Fake([30, 2], f)),
          dict(score=Fake([6, 2, 5], b)), dict(tok_start=Fake([3], i)), dict(block_tokens=40), dict(n_first=3), dict(n_last=-1),
          dict(max_new=2.5), dict(n_first=2 ** 40), dict(sel=Fake([6, 2, 3], i, "cuda:1")), dict(sel=Fake([6, 2, 0], i))]),
        (stq.stq_kv_attend_blocks, dict(kv=kv, table=table, tok_start=start, lens=lens, sel=sel, q=q, o=o, scale=0.1, max_new=2),
         [dict(sel=Fake([5, 2, 3], i)), dict(sel=Fake([6, 4, 3], i)), dict(sel=Fake([36], i)), dict(o=Fake([6, 4, 128], torch.float16)),
          dict(o=Fake([6, 2, 128], b)), dict(work=Fake([8], f)), dict(max_new=2 ** 32 + 1), dict(o=Fake([6, 4, 128], b, ptr=0x10010)),
          dict(sel=Fake([6, 2, 100], i, ptr=1 << 42))]),
        (stq.stq_kv_attend_shared, dict(kv=kv, table=table, tok_start=start, lens=lens, group_start=Fake([3], i), prefix=Fake([2], i), q=q, o=o,
                                        scale=0.1, max_new=2, max_own=100, max_prefix=128, work=big),
         [dict(group_start=Fake([2], i)), dict(prefix=Fake([2], torch.int64)), dict(work=Fake([1024], u, ptr=1 << 43)), dict(work=None),
          dict(max_prefix=-1), dict(max_own=0), dict(max_prefix=2 ** 31), dict(max_own=1.5), dict(group_start=Fake([3], i, "cuda:1"))]),
    ]
    for call, args, bad in calls:
        for kw in bad:
            with pytest.raises(E):
                call(**dict(args, **kw), stream=0)
        for name in args:
            if name not in ("kv", "max_new", "max_len", "scale", "block_tokens", "max_own", "max_prefix"):
                with pytest.raises(E):
                    call(**dict(args, **{name: None}), stream=0)
    with pytest.raises(E):
        stq.stq_kv_attend_blocks_bytes(kv, 3, 6, 4, 2 ** 31, 2)
    with pytest.raises(E):
        stq.stq_kv_attend_blocks_bytes(kv, 3, 6, 4, 1.5, 2)
    with pytest.raises(E):
        stq.stq_kv_attend_shared_bytes(kv, 3, 6, 4, 2, 2, 100, 2 ** 31)


def test_packed_descriptors_are_the_structures():
    from quantized_linear_attention_amd import _lib
    for pack, desc in ((_lib._select_desc, _lib._SelectDesc), (_lib._shared_desc, _lib._SharedDesc)):
        values = [3 + i for i, _ in enumerate(desc._fields_)]
        d = desc.from_buffer_copy(pack(*values))
        assert [getattr(d, n) for n, _ in desc._fields_] == values
