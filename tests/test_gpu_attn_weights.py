"""Softmax weights of concentrated rows: a few cached tokens far above all others (first tokens that
gather a row's attention), against binary64, for both attention kernels."""
import numpy as np
import pytest

import attn_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_amd as q
    return q


def cached(stq, K, V, T):
    """A cache of one request's keys and values [tokens][heads][d] and its table row."""
    import torch
    L, kv, d = K.shape
    nb = -(-L // T)
    cache = stq.make_kv(torch.full((stq.stq_kv_bytes(nb, T, kv, d),), 0xFF, dtype=torch.uint8, device="cuda"), T, kv, d)
    order = np.random.default_rng(L).permutation(nb)
    t = np.arange(L)
    slots = torch.as_tensor(order[t // T] * T + t % T, device="cuda")
    stq.stq_kv_store(cache, slots, torch.as_tensor(K, device="cuda").float(), torch.as_tensor(V, device="cuda").float())
    ko, vo = (torch.empty(L, kv, d, device="cuda") for _ in range(2))
    stq.stq_kv_fetch(cache, slots, ko, vo)
    table = torch.as_tensor(order[None], device="cuda", dtype=torch.int32)
    return cache, table, ko.double().cpu().numpy(), vo.double().cpu().numpy()


def attend(stq, cache, table, q, L, scale, max_len):
    import torch
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new, heads = q.shape[:2]
    o = torch.empty_like(q)
    size = stq.stq_kv_attend_bytes(cache, 1, new, heads, new, max_len)
    work = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
    stq.stq_kv_attend(cache, table, i32(0, new), i32(L), q, o, scale, new, max_len, work=work)
    torch.cuda.synchronize()
    return o.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gap", [12.5, 14.0, 16.6])
@pytest.mark.parametrize("d,new,heads,L", [(128, 1, 4, 16390), (64, 4, 6, 9000), (128, 20, 4, 16390), (64, 70, 1, 9000)])
def test_dominant_tokens(stq, dtype, gap, d, new, heads, L):
    """Four tokens `gap` nats above thousands of others, which together hold up to a twentieth of the row.

    Bound.  Weights are rounded to binary16, truncated for bfloat16 outputs: 2^-10 of a weight; where binary16 is
    subnormal, an absolute step of 2^-24 against at least 2^7 for the largest weight, 2^-31 of it.  The sum
    takes the same weights, so each moves the output by its share of v - o.  The logits' products: d sums in
    binary32 that may truncate, 2^-23 of sum |q k| each, two half steps of the logit and of the reference; exp2
    within 2^-22.  Sums of L terms in chains of L / 32 + 40 steps.  Last the output's own rounding."""
    import torch
    rng = np.random.default_rng(new)
    T = 64
    K, V = 0.05 * rng.standard_normal((L, 1, d)), 1 + 0.25 * rng.standard_normal((L, 1, d))
    top = np.arange(4) * 32 + 3                           # one for each wave of a workgroup that walks the whole request
    K[:, 0, :32] = 0
    K[top, 0] = 0
    K[top, 0, 5] = 6
    V[top] = 0
    cache, table, K, V = cached(stq, K, V, T)
    q = rng.standard_normal((new, heads, d))
    q[..., 5] = 4
    ty = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    qt = torch.as_tensor(q, device="cuda").to(ty)
    q = qt.double().cpu().numpy()
    scale = float(np.float32(gap / 24))
    for max_len in (1, L):                                # one part; as many as the length gives
        o = attend(stq, cache, table, qt, L, scale, max_len)
        for j in range(new):
            n = L - new + j + 1
            k, v = K[:n, 0], V[:n, 0]
            logit = scale * (q[j] @ k.T)                  # [heads][n]
            size = abs(scale) * (np.abs(q[j]) @ np.abs(k).T)
            w = np.exp(logit - logit.max(1, keepdims=True))
            tot = w.sum(1, keepdims=True)
            want = w @ v / tot
            err = d * 2.0 ** -23 * (size + size.max(1, keepdims=True)) + 4 * 2.0 ** -24 * 2 * np.abs(logit).max(1, keepdims=True)
            err = (err + 2.0 ** -21 + 2.0 ** -10) * w + 2.0 ** -31
            for h in range(heads):
                bound = (err[h] @ np.abs(v - want[h]) + (L / 32 + 40) * 2.0 ** -23 * (w[h] @ (np.abs(v) + np.abs(want[h])))) / tot[h]
                bound += R.HALF[dtype] * np.abs(want[h]) * 1.001 + 2.0 ** -25
                off = np.abs(o[j, h] - want[h])
                assert (off <= bound).all(), (max_len, j, h, (off / bound).max(), (off / np.abs(want[h])).max())


@pytest.mark.parametrize("dtype,mag,exp,scale", [("bf16", 100.0, 13, 0.088), ("bf16", 2.0 ** 100, 0, 0.088), ("bf16", 2.0 ** 100, 0, -0.088),
                                                 ("bf16", 2.0 ** 127, 13, 8.0), ("bf16", 2.0 ** -100, -23, 3e38),
                                                 ("fp16", 6e4, 13, 0.125), ("fp16", 6e4, 13, 30.0), ("fp16", 6e4, 13, -3e38)])
@pytest.mark.parametrize("d,new,heads,L", [(64, 1, 2, 700), (128, 6, 4, 1500), (128, 40, 2, 400), (64, 70, 1, 1500)])
def test_steep_rows(stq, dtype, mag, exp, scale, d, new, heads, L):
    """Logits of any finite size.  Two tokens with the same largest logit, all others below it by far
    more than a hundred: the output is the mean of the two's values (products, sums and the mean are exact;
    two binary32 steps for the quotient and the product with it, then the output's rounding)."""
    import torch
    rng = np.random.default_rng(d + new)
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    K = rng.choice([0.0, 0.5, 1.0, 1.5, 2.0], (L, 1, d)) * sign * np.where(rng.random((L, 1, d)) < 0.3, -1, 1)
    V = rng.standard_normal((L, 1, d))
    tops = np.array([37, 200])
    K[tops] = 4 * sign
    K[5], K[90] = 3 * sign, -6 * sign
    cache, table, K, V = cached(stq, K * 2.0 ** exp, V, 32)
    ty = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    for flip in (1.0, -1.0):                              # and the token with the most negative product on top
        q = torch.as_tensor(np.broadcast_to(sign * mag * np.sign(scale) * flip, (new, heads, d)).copy(), device="cuda").to(ty)
        top = tops if flip > 0 else np.array([90])
        for max_len in (1, L):
            o = attend(stq, cache, table, q, L, scale, max_len)
            want = V[top, 0].mean(0)
            assert np.isfinite(o).all()
            assert (np.abs(o - want) <= (R.HALF[dtype] + 2.0 ** -21) * np.abs(want) + 2.0 ** -25).all(), np.abs(o - want).max()
