"""Pins of the step oracle: hand-worked cases and planted mistakes (CPU)."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import step_oracle as S


def test_tables_by_hand():
    # sequence 0: 20 tokens, 2 pages held, 13 more -> 33 tokens, one page more;
    # sequence 1: idle; sequence 2: fits its page; sequence 3: a new request of 17.
    table = np.full((4, 4), -1)
    table[0, :2], table[2, :1] = [7, 3], [5]
    t, counts, left, q, new, pos, slots, codes = S.build_tables(
        [20, 4, 10, 0], [13, 0, 2, 17], table, [2, 1, 1, 0], [9, 8, 6, 1], 4, 34, 10)
    assert counts == [3, 1, 1, 2] and left == 1 and codes == set()
    assert q == [0, 13, 13, 15, 32] and new == [0, 1, 1, 1, 3]
    assert t[0, 2] == 1 and list(t[3, :2]) == [6, 8]          # the top of the stack first
    assert list(pos[:13]) == list(range(20, 33))
    assert list(slots[:13]) == [3 * 16 + i for i in range(4, 16)] + [16]
    assert list(slots[13:15]) == [5 * 16 + 10, 5 * 16 + 11]
    assert list(slots[15:32]) == [6 * 16 + i for i in range(16)] + [8 * 16]
    assert list(slots[32:]) == [-1, -1] and list(pos[32:]) == [0, 0]


def test_tables_run_out_in_order():
    # one page each wanted by 0 and 2, two by 1: with 2 free, 0 is served, 1 and
    # (being later) 2 are not
    t, counts, left, q, new, pos, slots, codes = S.build_tables(
        [0, 0, 0], [1, 17, 1], np.full((3, 2), -1), [0, 0, 0], [4, 5], 2, 19, 8)
    assert counts == [1, 0, 0] and left == 1 and new == [0, 1, 1, 1]
    assert slots[0] == 80 and set(slots[1:]) == {-1} and codes == {S.OUT_OF_PAGES}


def test_release_is_the_way_back():
    table = np.array([[4, 2, 9], [7, 1, -1]])
    counts, free, n, off, codes = S.release_pages([17, 0], table, [3, 2], [0, 0, 0, 0, 0], 1)
    assert counts == [2, 0] and n == 4 and off == [0, 1, 3] and free == [0, 9, 7, 1, 0]
    assert codes == set()
    counts, free, n, off, codes = S.release_pages([-1, 0], table, [3, 2], [0, 0], 1)
    assert counts == [3, 2] and n == 1 and codes == {S.BAD_LENGTH}


def test_rotation_closed_forms():
    x = np.zeros((2, 1, 64))
    x[:, 0, 0], x[:, 0, 8], x[:, 0, 40] = 1, 2, 5
    y = S.norm_rotate(x, None, 0, [math.pi / 2] + [0.0] * 7, None, [[1, 2]], False)
    # pair (0, 8): a quarter turn, then a half; the rest stays
    assert np.allclose(y[0, 0, [0, 8]], [-2, 1]) and np.allclose(y[1, 0, [0, 8]], [-1, -2])
    assert (y[:, 0, 40] == 5).all()
    x = np.random.default_rng(0).standard_normal((3, 2, 64))
    y = S.norm_rotate(x, np.ones(64), 0, np.geomspace(1, 1e-4, 32), None, [[3, 9, 70000]], True)
    assert np.allclose((y * y).mean(-1), 1)                  # a rotation keeps the norm
    # score of two rotated rows depends on the distance of their positions alone
    a = [S.norm_rotate(x[:1], None, 0, np.geomspace(1, 1e-4, 32), None, [[p]], False) for p in (5, 105)]
    b = [S.norm_rotate(x[1:2], None, 0, np.geomspace(1, 1e-4, 32), None, [[p]], False) for p in (9, 109)]
    assert np.allclose((a[0] * b[0]).sum(), (a[1] * b[1]).sum())


def test_axes_pick_their_positions():
    x = np.random.default_rng(1).standard_normal((1, 1, 64))
    f = [0.5] * 16
    both = S.norm_rotate(x, None, 0, f, [0, 1] * 8, [[3], [4]], False)
    for axis, p in ((0, 3), (1, 4)):
        one = S.norm_rotate(x, None, 0, f, None, [[p]], False)
        cols = [i for i in range(16) if i % 2 == axis] + [16 + i for i in range(16) if i % 2 == axis]
        assert np.array_equal(both[0, 0, cols], one[0, 0, cols])


def test_choice_by_hand():
    z = [[2.0, 1.9, 1.5, -1.0]] * 3
    # row 0 repeats nothing but its own token 0: 2 / 2 = 1, so 1.9 wins; row 1 adds
    # token 1: 1.9 / 2; row 2 adds token 2, whose 0.75 is the least of the seen
    out, pick = S.choose(z, [0, 3], [0, 1, 2], np.zeros((1, 4)), [2.0])
    assert list(pick) == [1, 2, 0]
    out, pick = S.choose(z[:1], [0, 1], [3], np.array([[-32768, 0, 0, 2]]), [2.0], [0.25], [0.5])
    assert list(out[0]) == [1.0, np.float32(1.9), 1.5, -2.0 - 1.5 - 0.25]   # -1*2, 3 counts
    out, pick = S.choose(z[:1], [0, 1], bias=[[(1, 5.0), (2, 9.0), (1, 0.5)]], mask=[[0b0011]])
    assert pick[0] == 1 and out[0, 1] == np.float32(np.float32(1.9) + np.float32(0.5))
    assert list(S.choose(z[:1], [0, 1], mask=[[0]])[1]) == [-1]
    assert list(S.choose(z[:1], [0, 1], mask=[[2]], mask_rows=[-1])[1]) == [0]
    assert list(S.choose([[np.nan, -np.inf, 3, 3]], [0, 1])[1]) == [2]      # lowest index of a tie


def test_history_by_hand():
    s = S.history(np.zeros((2, 64)), [5, 5, 9, 70, -1], [0, 3, 5], 64)
    assert s[0, 5] == 2 and s[0, 9] == 1 and s.sum() == 3
    s = S.history(s, [5, 9, 1, 1], [0, 2, 4], 64, accepted=[0, -1])
    assert s[0, 5] == 3 and s[0, 9] == 1 and s[1].sum() == 0
    s = S.history(s, [5, 3], [0, 2, 2], 64, prompt=True)
    assert s[0, 5] == 3 - 32768 and s[0, 3] == -32768
    s[0, 5] = 32767
    assert S.history(s, [5], [0, 1, 1], 64)[0, 5] == 32767


@pytest.mark.parametrize("plant", ["no block history", "mask off by one"])
def test_planted_mistakes_change_the_choice(plant):
    z = np.array([[2.0, 1.9, 1.5, -1.0]] * 2)
    right = S.choose(z, [0, 2], [0, 1], np.zeros((1, 4)), [2.0], mask=[[0b1111]] * 2)[1]
    if plant == "no block history":
        wrong = S.choose(z, [0, 2], [-1, -1], np.zeros((1, 4)), [2.0], mask=[[0b1111]] * 2)[1]
    else:
        wrong = S.choose(z, [0, 2], [0, 1], np.zeros((1, 4)), [2.0], mask=[[0b1101]] * 2)[1]
    assert list(right) != list(wrong)
