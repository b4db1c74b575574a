"""The references of the operators for long contexts against hand-worked values (no GPU)."""
import numpy as np
import pytest

import long_ref as L


def test_e5m2_rounds_outward():
    assert L.e5m2([1.0, 1.1, -1.1, 1.25, 1.26, 49152.0, 2.0 ** -16, 1e-9, -1e-9, 0.0], True).tolist() == \
        [1.0, 1.25, -1.0, 1.25, 1.5, 49152.0, 2.0 ** -16, 2.0 ** -16, 0.0, 0.0]
    assert L.e5m2([1.1, -1.1, -1e-9, 1e-9], False).tolist() == [1.0, -1.25, -2.0 ** -16, 0.0]


def test_e5m2_bytes_agree_with_torch():
    torch = pytest.importorskip("torch")
    raw = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(raw).view(torch.float8_e5m2).double().numpy()
    assert np.array_equal(L.e5m2_values(raw), want, equal_nan=True)
    fine = want[np.isfinite(want)]
    assert np.array_equal(L.e5m2(fine, True), fine) and np.array_equal(L.e5m2(fine, False), fine)


def test_touched_blocks():
    assert list(L.touched(65, 1, 64, 9, 1)) == [1] and list(L.touched(64, 1, 64, 9, 1)) == [0]
    assert list(L.touched(130, 70, 64, 9, 70)) == [0, 1, 2] and list(L.touched(130, 70, 64, 9, 4)) == [0]
    assert list(L.touched(5, 9, 64, 9, 9)) == [0] and list(L.touched(5, 0, 64, 9, 9)) == [] and list(L.touched(0, 0, 64, 9, 9)) == []
    assert list(L.touched(5, 9, 64, 9, 4)) == []          # the first four of them lie before position 0


def test_score_is_a_bound_and_the_best_corner():
    rng = np.random.default_rng(1)
    keys, x = rng.standard_normal((3, 20, 8)), rng.standard_normal((2, 8))
    b = np.stack([L.bounds(k) for k in keys])
    s, size = L.score(x, b)
    assert (s >= (keys @ x.T).max((1, 2))).all() and (size >= np.abs(s)).all()
    corner = max(sum(x[0, c] * b[0, (m >> c) & 1, c] for c in range(8)) for m in range(256))
    assert abs(L.score(x[:1], b)[0][0] - corner) < 1e-12


def test_select_by_hand():
    inf, nan = np.inf, np.nan
    s = np.array([1.0, 5.0, 5.0, -inf, 2.0, nan, 9.0, 0.0])
    assert L.select(s, 7 * 32 + 31, 32, 4, 0, 0) == [1, 2, 5, 6]
    assert L.select(s, 7 * 32, 32, 4, 1, 1) == [0, 5, 6, 7]
    assert L.select(s, 4 * 32, 32, 3, 0, 1) == [1, 2, 4]
    assert L.select(s, 4 * 32 + 5, 32, 2, 1, 0) == [0, 1]
    assert L.select(s, 3 * 32, 32, 6, 0, 0) == [0, 1, 2, -1, -1, -1]
    assert L.select(s, -1, 32, 2, 1, 1) == [-1, -1]


def test_listed_blocks():
    K, V = np.zeros((40, 32)), np.arange(40.0)[:, None] * np.ones(32)
    there = np.ones(40, bool)
    o, _ = L.attend_listed(np.ones(32), K, V, there, 35, [1, -1, 9], 32, 1.0, "bf16")
    assert np.allclose(o, 33.5)
    o, _ = L.attend_listed(np.ones(32), K, V, there, 32, [0, 1, 1], 32, 1.0, "bf16")
    assert np.allclose(o, (sum(range(32)) + 64) / 34)
    assert not L.attend_listed(np.ones(32), K, V, there, 20, [1], 32, 1.0, "bf16")[0].any()
