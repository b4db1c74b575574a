"""The plain references of the softmax layers' operators against hand-worked values (no GPU)."""
import numpy as np

import attn_ref as R


def test_levels_and_ties():
    x = np.zeros(32)
    x[:16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, .2500001]
    c, e = R.quantise(x)
    assert e.tolist() == [0]
    assert R.value(c, e)[:16].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, .5]


def test_exponents():
    want = {6: 0, 6.0001: 1, 3: -1, 3.0001: 0, 1e-30: -23, 1e30: 13, 0: 0, 6 * 2.0 ** 13: 13}
    assert {m: R.block_exp(m) for m in want} == want


def test_values_survive_requantisation():
    """Every value a block can hold next to its own largest code is stored as itself."""
    rng = np.random.default_rng(3)
    code = rng.integers(0, 16, (50, 64)).astype(np.uint8)
    code[:, 0], code[:, 32] = 7, 15
    e = rng.integers(-23, 14, (50, 2))
    x = R.value(code, e)
    assert np.array_equal(R.value(*R.quantise(x)), x)


def test_plan_by_hand():
    p = R.plan([31, 0, 64], [2, 0, 1], [9, 8], [[4, -1, -1], [-1] * 3, [5, 6, -1]], 32, 10, 5)
    assert p["table"].tolist() == [[4, 9, -1], [-1, -1, -1], [5, 6, 8]]
    assert p["tok_start"].tolist() == [0, 2, 2, 3] and p["lens"].tolist() == [33, 0, 65]
    assert p["pos"].tolist() == [31, 32, 64, -1, -1]
    assert p["slots"].tolist() == [4 * 32 + 31, 9 * 32, 8 * 32, -1, -1] and p["used"].tolist() == [2]


def test_attend_uniform_and_empty():
    K, V = np.zeros((5, 4)), np.arange(20.0).reshape(5, 4)
    o, _ = R.attend(np.ones((3, 4)), K, V, np.ones(5, bool), -1, 0.5, 2, 1, "bf16")
    assert o.tolist() == [[0, 0, 0, 0], V[0].tolist(), V[:2].mean(0).tolist()]
    o, _ = R.attend(np.ones((1, 4)), K, V, np.ones(5, bool), 4, 0.5, 2, 1, "bf16")
    assert np.allclose(o[0], V[[0, 3, 4]].mean(0))
