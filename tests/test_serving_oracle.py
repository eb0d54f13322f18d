"""Closed forms and invariants that pin oracle/serving.py (CPU only)."""
import math

import numpy as np
import pytest

from oracle import serving as S


def test_step_plan_worked_example():
    # request 0: 15 tokens + 2 -> one new page; 1: 16 + 1 -> one; 2: 3 + 0 -> none; 3: 0 + 33 -> 3
    table = np.full((4, 4), 99)
    table[0, 0], table[1, 0], table[2, 0] = 5, 6, 7
    r = S.step_plan([15, 16, 3, 0], [2, 1, 0, 33], table, [10, 11, 12, 13, 14, 15], 6, 20, 38)
    assert r["cu"].tolist() == [0, 2, 3, 3, 36]
    assert r["seq_lens"].tolist() == [17, 17, 3, 33]
    assert r["table"].tolist() == [[5, 15, 99, 99], [6, 14, 99, 99], [7, 99, 99, 99],
                                   [13, 12, 11, 99]]
    assert r["count"] == 1 and not r["flags"]
    assert r["slots"][:3].tolist() == [5 * 16 + 15, 15 * 16, 14 * 16]
    assert r["slots"][3] == 13 * 16 and r["slots"][35] == 11 * 16 and r["positions"][35] == 32
    assert r["slots"][36:].tolist() == [-1, -1]


def test_step_plan_serves_a_prefix_of_the_needs():
    # 2 free pages: 0 takes one, 1 needs two (waits), 2 needs none (served), 3 needs one (waits: the
    # pages asked for before it are gone)
    r = S.step_plan([0, 0, 4, 0], [1, 17, 2, 1], np.zeros((4, 2), int), [3, 4], 2, 9, 21)
    assert r["seq_lens"].tolist() == [1, 0, 6, 0] and r["count"] == 1
    assert r["flags"] == {"no_pages"}
    assert (r["slots"] >= 0).sum() == 3


def test_release_skips_entries_already_given_back():
    t, f, n, flags = S.release([0, 1], [3, 2], [[4, -1, 6], [7, 8, 9]], [1, 0, 0, 0, 0], 1, 10)
    assert t.tolist() == [[-1, -1, -1], [7, -1, 9]]
    assert f[:4].tolist() == [1, 4, 6, 8] and n == 4 and not flags
    t, f, n, flags = S.release([0], [3], [[4, 5, 6]], [1, 0], 1, 10)
    assert t.tolist() == [[4, 5, 6]] and n == 1 and flags == {"length"}


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_by_the_distance(interleaved):
    rng = np.random.default_rng(3)
    f = 1e4 ** (-np.arange(64) / 64)
    x, y = rng.standard_normal((2, 1, 1, 128))
    turn = lambda v, p: S.rope_rows(v, [p], f, interleaved)[0, 0]
    assert np.allclose(turn(x, 0), x[0, 0])
    assert np.isclose(np.linalg.norm(turn(x, 77)), np.linalg.norm(x))
    # the product of two rotated rows depends on the difference of their positions alone
    assert np.isclose(turn(x, 900) @ turn(y, 893), turn(x, 7) @ turn(y, 0))


def test_rope_quarter_turn_pairs():
    x = np.arange(16.0).reshape(1, 1, 16)
    f = np.zeros(4)
    f[1] = math.pi / 2
    half = S.rope_rows(x, [1], f, False)[0, 0]
    assert np.allclose(half[[1, 5]], [-5, 1]) and np.allclose(np.delete(half, [1, 5]),
                                                             np.delete(np.arange(16.0), [1, 5]))
    inter = S.rope_rows(x, [1], f, True)[0, 0]
    assert np.allclose(inter[[2, 3]], [-3, 2])


def test_visible_sets():
    assert S.visible(3, 6).tolist() == [1, 1, 1, 1, 0, 0]
    assert S.visible(3, 6, window=2).tolist() == [0, 0, 1, 1, 0, 0]
    assert S.visible(3, 6, window=2, prefix=1).tolist() == [1, 0, 1, 1, 0, 0]
    assert S.visible(1, 6, prefix=4).tolist() == [1, 1, 1, 1, 0, 0]
    assert S.visible(3, 6, row_start=3).tolist() == [0, 0, 0, 1, 0, 0]
    assert S.visible(3, 6, row_start=4).tolist() == [0] * 6
    assert S.visible(3, 6, row_start=9, prefix=99).tolist() == [1] * 6


def test_attend_scored_closed_forms():
    rng = np.random.default_rng(5)
    K, V = rng.standard_normal((2, 9, 4))
    q = rng.standard_normal(4)
    # one visible key: its value, whatever the cap and the bias
    o, l = S.attend_scored(q, K, V, 8, S.visible(8, 9, window=1), 0.5, 3.0, 0.7)
    assert np.allclose(o, V[8]) and np.isclose(l, 3 * math.tanh(0.5 * (K[8] @ q) / 3))
    # equal scores under a bias: weights are a geometric series in the distance
    o, l = S.attend_scored(0 * q, K, V, 8, S.visible(8, 9), 1.0, 0.0, math.log(2))
    w = 0.5 ** np.arange(8, -1, -1)
    assert np.allclose(o, w @ V / w.sum()) and np.isclose(l, math.log(w.sum()))
    # a cap far above the scores changes nothing; a tiny cap makes all keys equal
    plain = S.attend_scored(q, K, V, 8, S.visible(8, 9), 1.0)
    assert np.allclose(S.attend_scored(q, K, V, 8, S.visible(8, 9), 1.0, 1e6)[0], plain[0], atol=1e-9)
    assert np.allclose(S.attend_scored(q, K, V, 8, S.visible(8, 9), 1.0, 1e-9)[0], V.mean(0))
    # nothing visible
    o, l = S.attend_scored(q, K, V, 8, np.zeros(9, bool), 1.0)
    assert not o.any() and l == -math.inf
