"""Measured cases of the operators that serve long contexts over the 4-bit key/value cache: per-block bounds of the
keys, the blocks' scores for a query, the selection by them and attention over the selected blocks; attention for
requests that share a prefix.

`run` computes an operator in its plain form (elementary torch operations in binary32), or through the
library where `own` is true.
"""
import math
import random

import numpy as np
import torch

own = False

BF16, FP16 = "bf16", "fp16"
_TYPES = {BF16: torch.bfloat16, FP16: torch.float16}
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # magnitudes of the 3-bit code; bit 3 is the sign
_E_MIN, _E_MAX = -23, 13                                # exponents of the 32-channel scales
_MOST = 1 << 26                                         # channels quantised at a time


def listed():
    return [
        # one decode step: the block that each request's token went to
        dict(name="bounds_decode", op="bounds", n=512, ctx=8191, new=1, kv_heads=8, d=128, block=64),
        # a batch of prompts: all their blocks
        dict(name="bounds_prompt", op="bounds", n=4, ctx=9001, new=8192, kv_heads=8, d=128, block=64),
        # one decode step's scores over long contexts
        dict(name="score_decode", op="score", n=64, ctx=32768, new=1, heads=32, kv_heads=8, d=128, block=64, dtype=BF16),
        # every token of two prompts scores the blocks behind it
        dict(name="score_prompt", op="score", n=2, ctx=16384, new=2048, heads=32, kv_heads=8, d=128, block=64, dtype=BF16),
        # the selection of that decode step, and of those prompts
        dict(name="select_decode", op="select", n=64, ctx=32768, new=1, kv_heads=8, block=64, top=64, first=1, last=2),
        dict(name="select_prompt", op="select", n=2, ctx=16384, new=2048, kv_heads=8, block=64, top=32, first=1, last=1),
        # one request with a long context: latency
        dict(name="blocks_single", op="blocks", n=1, ctx=131072, new=1, heads=32, kv_heads=8, d=128, block=64, top=32,
             dtype=BF16),
        # a serving batch's decode step, 4,096 tokens of each request's context
        dict(name="blocks_batch", op="blocks", n=64, ctx=32768, new=1, heads=32, kv_heads=8, d=128, block=64, top=64,
             dtype=BF16),
        # a prompt over what is cached already, each token with its own blocks
        dict(name="blocks_prompt", op="blocks", n=1, ctx=8192, new=1021, heads=32, kv_heads=4, d=64, block=64, top=16,
             dtype=FP16),
        # a few requests behind one system prompt
        dict(name="shared_small", op="shared", groups=1, members=8, prefix=2048, own=512, new=1, heads=32, kv_heads=8,
             d=128, block=64, dtype=BF16),
        # a serving batch's decode step: two prompts, 32 requests or fewer each
        dict(name="shared_batch", op="shared", groups=2, members=32, prefix=8192, own=1024, new=1, heads=32, kv_heads=8,
             d=128, block=64, dtype=BF16),
        # drafted tokens of many requests behind four long prompts
        dict(name="shared_draft", op="shared", groups=4, members=64, prefix=16384, own=2048, new=4, heads=32, kv_heads=8,
             d=128, block=64, dtype=BF16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["bounds", "score", "select", "blocks", "blocks", "shared", "shared"])
    block = rng.choice([32, 64, 128])
    d = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 5, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 6, 8, 16])
    c = dict(op=op, kv_heads=kv, block=block)
    if op == "shared":
        groups = rng.choice([1, 1, 2, 3, 5])
        new = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 200)])
        prefix = _log(rng, block, 32768)
        room = 256 * 4 * 32 * 16384 * 128 / (groups * new * heads * (prefix + 1024) * d)
        return dict(c, groups=groups, members=_log(rng, 1, max(1, min(128, int(room)))), prefix=prefix,
                    own=new + _log(rng, 1, 2048), new=new, heads=heads, d=d, dtype=rng.choice([BF16, FP16]))
    new = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
    ctx = new + _log(rng, 1, 65536 if new > 8 else 131072)
    if op == "bounds":
        return dict(c, n=_log(rng, 1, max(1, min(512, 65536 // new, (1 << 22) // (ctx * kv)))), ctx=ctx, new=new, d=d)
    if op == "score":
        n = _log(rng, 1, max(1, min(256, (1 << 24) // (new * kv * (ctx // block + 1)))))
        return dict(c, n=n, ctx=ctx, new=new, heads=heads, d=d, dtype=rng.choice([BF16, FP16]))
    top = _log(rng, 2, 128)
    if op == "select":                                   # from contexts of many more blocks than are selected
        ctx = max(ctx, new + 32 * block)
        n = _log(rng, 1, max(1, min(256, (1 << 24) // (new * kv * (ctx // block + 1)))))
        return dict(c, n=n, ctx=ctx, new=new, top=min(top + 6, ctx // block // 4), first=rng.randint(0, 2),
                    last=rng.randint(0, 3))
    new = min(new, max(1, (1 << 24) // (kv * top * block)))
    n = _log(rng, 1, max(1, min(128, (1 << 22) // (ctx * kv), (1 << 24) // (new * kv * top * block))))
    return dict(c, n=n, ctx=ctx, new=new, heads=heads, d=d, top=top, dtype=rng.choice([BF16, FP16]))


# ------------------------------------------------------------------- sizes

def _counts(c):
    """Cached and new tokens of each request: ragged, the first the longest; the same for every seed."""
    r = random.Random("%d %d %d" % (c["n"], c["ctx"], c["new"]))
    new = [c["new"] if i == 0 else r.randint((c["new"] + 1) // 2, c["new"]) for i in range(c["n"])]
    top = c["ctx"] - c["new"]
    return [top if i == 0 else r.randint(top // 4, top) for i in range(c["n"])], new


def _groups(c):
    """(members, prefix) of each group and the own tokens, new ones among them, and new tokens of each request."""
    r = random.Random("%d %d %d" % (c["members"], c["prefix"], c["own"]))
    T = c["block"]
    size, prefix, mine, new = [], [], [], []
    for g in range(c["groups"]):
        size.append(c["members"] if g == 0 else r.randint((c["members"] + 1) // 2, c["members"]))
        prefix.append((c["prefix"] if g == 0 else r.randint(c["prefix"] // 2, c["prefix"])) // T * T)
        for i in range(size[g]):
            new.append(c["new"] if i == 0 else r.randint((c["new"] + 1) // 2, c["new"]))
            mine.append(c["own"] if g == i == 0 else r.randint(new[-1], c["own"]))
    return size, prefix, mine, new


def work(c):
    T, kv = c["block"], c["kv_heads"]
    if c["op"] == "shared":
        size, prefix, mine, new = _groups(c)
        head = [p for p, m in zip(prefix, size) for _ in range(m)]
        pairs = sum(m * (p + own - m) + m * (m + 1) // 2 for p, own, m in zip(head, mine, new))
        return {"bytes": (sum(prefix) + sum(mine)) * kv * c["d"] * 17 // 16 + 4 * sum(new) * c["heads"] * c["d"],
                "flops": 4 * c["d"] * c["heads"] * pairs}
    old, new = _counts(c)
    if c["op"] == "bounds":
        d, cols = c["d"], sum((a + b - 1) // T - a // T + 1 for a, b in zip(old, new))
        tokens = sum(a + b - a // T * T for a, b in zip(old, new))
        return {"bytes": kv * (tokens * (d // 2 + d // 32) + cols * 2 * d), "flops": 2 * kv * tokens * d}
    seen = [sum((a + j) // T + 1 for j in range(b)) for a, b in zip(old, new)]          # (token, block) pairs
    if c["op"] == "score":
        once = sum((a + b - 1) // T + 1 for a, b in zip(old, new))
        return {"bytes": kv * (once * 2 * c["d"] + sum(seen) * 4) + 2 * sum(new) * c["heads"] * c["d"],
                "flops": 4 * c["d"] * c["heads"] * sum(seen)}
    if c["op"] == "select":
        return {"bytes": kv * 4 * (sum(seen) + sum(new) * c["top"]), "flops": 0}
    # each listed block once for each token and head, where the request has as many bytes; else all it has
    tokens = pairs = 0
    for a, b in zip(old, new):
        mine = [min(a + j + 1, (min(c["top"], (a + j) // T + 1) - 1) * T + (a + j) % T + 1) for j in range(b)]
        pairs += sum(mine)
        tokens += min(sum(mine), a + b)
    return {"bytes": kv * (tokens * c["d"] * 17 // 16 + 4 * sum(new) * c["top"]) + 4 * sum(new) * c["heads"] * c["d"],
            "flops": 4 * c["d"] * c["heads"] * pairs}


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """Codes (0..15) and scale exponents of x [..., d] in blocks of 32 channels."""
    y = x.float().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1)
    m, ex = torch.frexp(top)
    e = torch.where(m <= 0.75, ex - 3, ex - 2)           # least e with top <= 6 * 2^e
    e = torch.where(top == 0, torch.zeros_like(e), e.clamp(_E_MIN, _E_MAX))
    a = torch.ldexp(y.abs(), -e.unsqueeze(-1))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + (torch.signbit(y) & (code > 0)).to(torch.uint8) * 8
    return code.flatten(-2), e


def _pages(blocks, c, gen):
    """Pages [blocks][heads][bytes] of tokens as a projection and a norm leave them: channels of unit size with a few
    large ones, and a mean of their own in each key channel."""
    kv, d, T = c["kv_heads"], c["d"], c["block"]
    pages = torch.zeros(blocks, kv, T * d * 17 // 16, dtype=torch.uint8, device="cuda")
    size = torch.exp(0.5 * torch.randn(kv, 1, d, device="cuda", generator=gen))
    mean = 0.5 * torch.randn(kv, 1, d, device="cuda", generator=gen)
    step = max(1, _MOST // (kv * T * d))
    for b in range(0, blocks, step):
        part = pages[b: b + step]
        for at in (0, 1):
            x = torch.randn(part.shape[0], kv, T, d, device="cuda", generator=gen)
            if at == 0:                                  # blocks differ in their means too: what a score tells apart
                x = 0.8 * x + mean + 0.6 * torch.randn(part.shape[0], kv, 1, d, device="cuda", generator=gen)
            code, e = _quantise(x * size)
            part[..., at * (T * d // 2): (at + 1) * (T * d // 2)] = (code[..., 0::2] | (code[..., 1::2] << 4)).flatten(-2)
            s = T * d + at * (T * d // 32)
            part[..., s: s + T * d // 32] = (e + 127).to(torch.uint8).transpose(-1, -2).flatten(-2)
    return pages


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device="cuda")
    st = dict(case=dict(c))
    T, kv = c["block"], c["kv_heads"]
    if c["op"] == "shared":
        size, prefix, mine, new = _groups(c)
        head = [p for p, m in zip(prefix, size) for _ in range(m)]
        lens = [p + m for p, m in zip(head, mine)]
        st.update(group_start=torch.tensor(np.cumsum([0] + size), **i32), prefix=torch.tensor(prefix, **i32))
    else:
        old, new = _counts(c)
        lens = [a + b for a, b in zip(old, new)]
        head = [0] * len(lens)
    n, tok, cols = len(lens), sum(new), max(-(-m // T) for m in lens)
    blocks = sum(-(-(m - h) // T) for m, h in zip(lens, head)) + sum(st["prefix"].tolist() if c["op"] == "shared" else []) // T + 7
    ids = torch.randperm(blocks, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((n, cols), -1, **i32)
    at, first = 0, -1
    starts = set(st["group_start"].tolist()[:-1]) if c["op"] == "shared" else ()
    for i, (m, h) in enumerate(zip(lens, head)):
        if i in starts:                                  # the group's first request brings the prefix' blocks
            table[i, : h // T] = ids[at: at + h // T]
            at, first = at + h // T, i
        elif h:
            table[i, : h // T] = table[first, : h // T]
        nb = -(-(m - h) // T)
        table[i, h // T: h // T + nb] = ids[at: at + nb]
        at += nb
    st.update(table=table, lens=torch.tensor(lens, **i32), tok_start=torch.tensor(np.cumsum([0] + new), **i32),
              blocks=blocks, tok=tok)
    if c["op"] in ("bounds", "blocks", "shared"):
        st["pages"] = _pages(blocks, c, gen)
    if c["op"] == "bounds":                               # (one block more: where the plain form puts what has no place)
        st["spare"] = torch.zeros(blocks + 1, kv, 2, c["d"], dtype=torch.uint8, device="cuda")
        st["bounds"] = st["spare"][:blocks].view(torch.float8_e5m2)
        return st
    if c["op"] != "select":
        dt = _TYPES[c["dtype"]]
        q = torch.randn(tok, c["heads"], c["d"], device="cuda", generator=gen)
        st.update(q=q.to(dt), scale=c["d"] ** -0.5)
    if c["op"] == "score":
        mean = torch.randn(blocks, kv, 1, c["d"], device="cuda", generator=gen)
        reach = 2 + torch.rand(blocks, kv, 2, c["d"], device="cuda", generator=gen)
        sign = torch.tensor([-1.0, 1.0], device="cuda")[:, None]
        st.update(bounds=(mean + sign * reach).to(torch.float8_e5m2), pages=torch.zeros(blocks, kv, T * c["d"] * 17 // 16,
                  dtype=torch.uint8, device="cuda"), score=torch.full((tok, kv, cols), -math.inf, device="cuda"))
    elif c["op"] == "select":                            # (rounded: some are equal)
        st.update(score=(8 + 4 * torch.randn(tok, kv, cols, device="cuda", generator=gen)).half().float(),
                  sel=torch.full((tok, kv, c["top"]), -1, **i32))
    else:
        st["o"] = torch.zeros_like(st["q"])
    if c["op"] == "blocks":                              # the first block, the last one, and any others
        last = torch.cat([torch.arange(a, a + b) for a, b in zip(old, new)]).cuda()[:, None, None] // T
        order = torch.rand(tok, kv, cols, device="cuda", generator=gen)
        col = torch.arange(cols, device="cuda")
        order = torch.where((col == 0) | (col == last), order + 2, order).masked_fill_(col > last, -1)
        best = order.sort(-1, descending=True)
        if cols < c["top"]:
            best = [torch.nn.functional.pad(x, (0, c["top"] - cols), value=-1) for x in best]
        at = torch.where(best[0][..., : c["top"]] < 0, cols, best[1][..., : c["top"]]).sort(-1)[0]
        st["sel"] = torch.where(at == cols, -1, at).to(torch.int32).contiguous()
    return st


# -------------------------------------------------------------- plain forms

def _values(page, part, T, d):
    """Keys (part 0) or values (part 1) of pages [..., bytes] in binary32: [..., T, d]."""
    lut = torch.tensor(_LEVELS + tuple(-x for x in _LEVELS), device=page.device)
    pair = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)
    code = page[..., part * (T * d // 2): (part + 1) * (T * d // 2)].unflatten(-1, (T, d // 2))
    at = T * d + part * (T * d // 32)
    sc = (page[..., at: at + T * d // 32].int() << 23).view(torch.float32).unflatten(-1, (d // 32, T)).transpose(-1, -2)
    return (pair[code.int()].flatten(-2).unflatten(-1, (d // 32, 32)) * sc[..., None]).flatten(-2)


def _upward(x, up):
    """Binary16 numbers x as the upper bytes of the next ones at or above (below) them that have no other bits."""
    u = x.half().view(torch.int16).int() & 0xFFFF
    away = ((u & 0xFF) > 0) & ((u < 0x8000) == up)
    return ((u >> 8) + away).to(torch.uint8)


def _bounds(s):
    c = s["case"]
    T, d = c["block"], c["d"]
    lens, base = s["lens"].long(), s["lens"].long() - (s["tok_start"][1:] - s["tok_start"][:-1]).long()
    col = base[:, None] // T + torch.arange((c["new"] - 1) // T + 2, device="cuda")       # [n][touched]
    on = col * T < lens[:, None]
    blk = torch.where(on, s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)), s["blocks"]).long()
    K = _values(s["pages"][blk.clamp(max=s["blocks"] - 1)], 0, T, d)                       # [n][touched][kv][T][d]
    there = (col[..., None] * T + torch.arange(T, device="cuda") < lens[:, None, None])[:, :, None, :, None]
    lo = K.masked_fill(~there, math.inf).amin(-2)
    hi = K.masked_fill(~there, -math.inf).amax(-2)
    s["spare"][blk] = torch.stack([_upward(lo, False), _upward(hi, True)], -2)
    return s["bounds"]


def _rows(s, r):
    """Query rows [n][kv][r * new][d] (head-major), positions [n][new], and each token's (request, query)."""
    kv, new = s["case"]["kv_heads"], s["case"]["new"]
    lens, starts = s["lens"].long(), s["tok_start"].long()
    j = torch.arange(new, device="cuda")[None]
    row = (starts[:-1, None] + j).clamp(max=s["tok"] - 1)
    Q = s["q"].float()[row].unflatten(2, (kv, r)).permute(0, 2, 3, 1, 4).flatten(2, 3) if r else None
    t = torch.arange(s["tok"], device="cuda")
    i = torch.searchsorted(starts[1:], t, right=True)
    return Q, (lens - (starts[1:] - starts[:-1]))[:, None] + j, i, t - starts[i]


def _score(s):
    c = s["case"]
    kv, r = c["kv_heads"], c["heads"] // c["kv_heads"]
    Q, p, i, j = _rows(s, r)
    B = s["bounds"].view(torch.uint8)[s["table"].long().clamp(min=0)].view(torch.float8_e5m2).float().transpose(1, 2)
    lo, hi = B[..., 0, :].transpose(-1, -2), B[..., 1, :].transpose(-1, -2)               # [n][kv][d][cols]
    Q = Q * s["scale"]
    S = (torch.matmul(Q.clamp(min=0), hi) + torch.matmul(Q.clamp(max=0), lo)).unflatten(2, (r, c["new"])).amax(2)
    see = torch.arange(S.shape[-1], device="cuda") * c["block"] <= p[..., None]
    return S.masked_fill(~see[:, None], -math.inf).transpose(1, 2)[i, j].contiguous()


def _select(s):
    c = s["case"]
    _, p, i, j = _rows(s, 0)
    last = (p[i, j] // c["block"])[:, None, None]
    x = s["score"]
    col = torch.arange(x.shape[-1], device="cuda")
    must = (col <= last) & ((col < c["first"]) | (col > last - c["last"]))
    rank = torch.where(must, 2, ((col <= last) & (x != -math.inf)).int())
    order = x.sort(dim=-1, descending=True, stable=True)[1]
    order = order.gather(-1, rank.gather(-1, order).sort(dim=-1, descending=True, stable=True)[1])[..., : c["top"]]
    at = torch.where(rank.gather(-1, order) > 0, order, x.shape[-1]).sort(-1)[0]
    at = torch.where(at == x.shape[-1], -1, at).to(torch.int32)
    return torch.nn.functional.pad(at, (0, c["top"] - at.shape[-1]), value=-1)


def _blocks(s):
    c = s["case"]
    T, d, kv = c["block"], c["d"], c["kv_heads"]
    _, p, i, j = _rows(s, 0)
    sel = s["sel"].long()
    blk = s["table"].long()[i[:, None, None], sel.clamp(min=0)]
    page = s["pages"][blk, torch.arange(kv, device="cuda")[:, None]]                       # [tok][kv][top][bytes]
    Q = s["q"].float().unflatten(1, (kv, -1))
    S = torch.matmul(Q, _values(page, 0, T, d).flatten(2, 3).transpose(-1, -2)) * s["scale"]
    see = (sel[..., None] * T + torch.arange(T, device="cuda") <= p[i, j][:, None, None, None]) & (sel[..., None] >= 0)
    S = S.masked_fill(~see.flatten(2)[:, :, None], -math.inf)
    w = torch.exp(S - S.amax(-1, keepdim=True))
    O = torch.matmul(w, _values(page, 1, T, d).flatten(2, 3)) / w.sum(-1, keepdim=True)
    return O.flatten(1, 2).to(s["q"].dtype)


def _shared(s):
    c = s["case"]
    T, d, kv, new = c["block"], c["d"], c["kv_heads"], c["new"]
    r = c["heads"] // kv
    Q, p, i, j = _rows(s, r)
    first, n, cols = s["group_start"].long(), Q.shape[0], s["table"].shape[1]
    req = torch.arange(n, device="cuda")
    g = torch.searchsorted(first[1:], req, right=True)                                     # the request's group
    prefix = s["prefix"].long()
    # the prefix: all rows of a group against its blocks, which are read once
    wide = c["prefix"] // T
    page = s["pages"][s["table"].long()[first[:-1], :wide].clamp(min=0)].transpose(1, 2)   # [groups][kv][wide][bytes]
    K, V = (_values(page, part, T, d).flatten(2, 3) for part in (0, 1))
    most = c["members"]
    mine = (first[:-1, None] + torch.arange(most, device="cuda")).clamp(max=n - 1)         # [groups][members]
    rows = Q[mine].transpose(1, 2).flatten(2, 3)                                           # [groups][kv][members * r * new][d]
    S = torch.matmul(rows, K.transpose(-1, -2)) * s["scale"]
    S = S.masked_fill_((torch.arange(wide * T, device="cuda") >= prefix[:, None])[:, None, None], -math.inf)
    # each request's own tokens
    col = prefix[g][:, None] // T + torch.arange((c["own"] - 1) // T + 1, device="cuda")
    page = s["pages"][s["table"].long().gather(1, col.clamp(max=cols - 1)).clamp(min=0)].transpose(1, 2)
    Ko, Vo = (_values(page, part, T, d).flatten(2, 3) for part in (0, 1))
    t = (col[..., None] * T + torch.arange(T, device="cuda")).flatten(1)[:, None]           # [n][1][own tokens]
    So = (torch.matmul(Q, Ko.transpose(-1, -2)) * s["scale"]).unflatten(2, (r, new))
    So = So.masked_fill_(~(t <= p[..., None])[:, None, None], -math.inf).flatten(2, 3)      # [n][kv][r * new][own]
    # one softmax over both
    m1, m2 = S.amax(-1, keepdim=True), So.amax(-1, keepdim=True)
    here = req - first[g]
    top = torch.maximum(m1.unflatten(2, (most, r * new))[g, :, here], m2)                   # [n][kv][r * new][1]
    back = torch.zeros(mine.shape + top.shape[1:], device="cuda").index_put((g, here), top)
    S = S.sub_(back.transpose(1, 2).flatten(2, 3)).exp_()
    So = So.sub_(top).exp_()
    O = torch.matmul(S, V).unflatten(2, (most, r * new))[g, :, here] + torch.matmul(So, Vo)
    O = O / (S.sum(-1, keepdim=True).unflatten(2, (most, r * new))[g, :, here] + So.sum(-1, keepdim=True))
    O = O.unflatten(2, (r, new)).permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["q"].dtype)      # [n][new][heads][d]
    return O[i, j]


def _own(s):
    import quantized_linear_attention_amd as stq
    c = s["case"]
    if c["op"] == "select":
        stq.stq_kv_select(s["score"], s["tok_start"], s["lens"], s["sel"], block_tokens=c["block"], max_new=c["new"],
                          n_first=c["first"], n_last=c["last"])
        return s["sel"]
    kv = stq.make_kv(s["pages"], c["block"], c["kv_heads"], c["d"])
    if c["op"] == "bounds":
        stq.stq_kv_bounds(kv, s["table"], s["tok_start"], s["lens"], s["bounds"], max_new=c["new"])
        return s["bounds"]
    if c["op"] == "score":
        stq.stq_kv_score(kv, s["bounds"], s["table"], s["tok_start"], s["lens"], s["q"], s["score"], scale=s["scale"],
                         max_new=c["new"], max_len=c["ctx"])
        return s["score"]
    n = s["lens"].shape[0]
    if c["op"] == "blocks":
        if "work" not in s:                               # the program's own workspace
            size = stq.stq_kv_attend_blocks_bytes(kv, n, s["tok"], c["heads"], c["top"], c["new"])
            s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        stq.stq_kv_attend_blocks(kv, s["table"], s["tok_start"], s["lens"], s["sel"], s["q"], s["o"], scale=s["scale"],
                                 max_new=c["new"], work=s["work"])
        return s["o"]
    if "work" not in s:
        size = stq.stq_kv_attend_shared_bytes(kv, n, s["tok"], c["heads"], c["groups"], c["new"], c["own"], c["prefix"])
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    stq.stq_kv_attend_shared(kv, s["table"], s["tok_start"], s["lens"], s["group_start"], s["prefix"], s["q"], s["o"],
                             scale=s["scale"], max_new=c["new"], max_own=c["own"], max_prefix=c["prefix"], work=s["work"])
    return s["o"]


def run(s):
    if own:
        return _own(s)
    return dict(bounds=_bounds, score=_score, select=_select, blocks=_blocks, shared=_shared)[s["case"]["op"]](s)


# ------------------------------------------------------------------- exact

def _two(e):
    """2^e in binary64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_page(byte, scale):
    """byte [m][d/2], scale [m][d/32] -> [m][d] in binary64, from the code's sign, exponent and mantissa bits."""
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).double()
    sign = 1 - 2 * torch.floor(code / 8)
    mag = code % 8
    ex, man = torch.floor(mag / 2), mag % 2
    val = torch.where(ex > 0, (1 + man / 2) * 2 ** (ex - 1), man / 2)
    return sign * val * _two(scale.long() - 127).repeat_interleave(32, 1)


def _exact_request(s, i, h, part):
    """Keys (part 0) or values (1) of request i and head h in binary64: [length][d]."""
    c, m = s["case"], int(s["lens"][i])
    T, d = c["block"], c["d"]
    pg = s["pages"][s["table"][i, : -(-m // T)].long(), h]
    byte = pg[:, part * T * d // 2: (part + 1) * T * d // 2].reshape(-1, d // 2)
    at = T * d + part * (T * d // 32)
    return _exact_page(byte, pg[:, at: at + T * d // 32].reshape(-1, d // 32, T).transpose(1, 2).reshape(-1, d // 32))[:m]


def _grid(x, up):
    """The nearest numbers at or above (below) x with three significant bits, no finer than 2^-16."""
    step = _two(torch.frexp(x.abs().clamp(min=2.0 ** -14))[1] - 3)
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def exact(c, seed):
    s = prepare(c, seed)
    T, kv = c["block"], c["kv_heads"]
    starts, lens = s["tok_start"].tolist(), s["lens"].tolist()
    base = [m - (b - a) for m, a, b in zip(lens, starts, starts[1:])]
    if c["op"] == "bounds":
        out = torch.zeros(s["bounds"].shape, dtype=torch.float64, device="cuda")
        for i, m in enumerate(lens):
            for h in range(kv):
                first = base[i] // T * T
                K = _exact_request(s, i, h, 0)[first:]
                for b in range(-(-K.shape[0] // T)):
                    x = K[b * T: (b + 1) * T]
                    to = out[int(s["table"][i, first // T + b]), h]
                    to[0], to[1] = _grid(x.amin(0), False), _grid(x.amax(0), True)
        return out
    if c["op"] == "select":
        x, out = s["score"].cpu().numpy(), np.full(s["sel"].shape, -1, np.int32)
        at = 0
        for i in range(len(lens)):
            for p in range(base[i], lens[i]):
                nb = p // T + 1
                b = np.arange(nb)
                must = (b < c["first"]) | (b >= nb - c["last"])
                for h in range(kv):
                    order = np.lexsort((b, -x[at, h, :nb], ~must))[: c["top"]]
                    out[at, h, : order.size] = np.sort(order)
                at += 1
        return out
    r, d = c["heads"] // kv, c["d"]
    if c["op"] == "score":
        out = torch.full(s["score"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for i, m in enumerate(lens):
            nb = -(-m // T)
            B = s["bounds"].view(torch.uint8)[s["table"][i, :nb].long()].view(torch.float8_e5m2).double()
            see = torch.arange(nb, device="cuda") * T <= torch.arange(base[i], m, device="cuda")[:, None]
            for h in range(kv):
                X = s["q"][starts[i]: starts[i + 1], h * r: (h + 1) * r].double() * s["scale"]
                best = torch.full(see.shape, -math.inf, dtype=torch.float64, device="cuda")
                for g in range(r):
                    x = X[:, g]
                    mid, half = (B[:, h, 0] + B[:, h, 1]) / 2, (B[:, h, 1] - B[:, h, 0]) / 2
                    best = torch.maximum(best, x @ mid.T + x.abs() @ half.T)
                out[starts[i]: starts[i + 1], h, :nb] = best.masked_fill(~see, -math.inf)
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, m in enumerate(lens):
        see = torch.arange(m, device="cuda")[None] <= torch.arange(base[i], m, device="cuda")[:, None]
        for h in range(kv):
            K, V = _exact_request(s, i, h, 0), _exact_request(s, i, h, 1)
            on = see
            if c["op"] == "blocks":
                sel = s["sel"][starts[i]: starts[i + 1], h].long()
                held = torch.zeros(sel.shape[0], s["table"].shape[1] + 1, dtype=torch.bool, device="cuda")
                held.scatter_(1, torch.where(sel < 0, held.shape[1] - 1, sel), True)
                on = see & held[:, :-1].repeat_interleave(T, 1)[:, :m]
            for g in range(h * r, (h + 1) * r):
                x = s["q"][starts[i]: starts[i + 1], g].double()
                out[starts[i]: starts[i + 1], g] = torch.softmax((x @ K.T * s["scale"]).masked_fill(~on, -math.inf), -1) @ V
    return out
