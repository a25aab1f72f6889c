"""Served block lengths of a table build: the oracle by hand, the argument errors of
the C entry, and why a step needs them (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import splash_oracle as O
from oracle import step_oracle as S

from test_capi_step_host import F, TABLES, TABLES_OK, call, lib  # noqa: F401


def test_oracle_by_hand():
    # pages for 0 and 3 of four, 1 needs none, 2 needs two of the one that is left
    table = np.full((4, 3), -1)
    table[1, 0] = 9
    served = []
    t, counts, left, q, new, pos, slots, codes = S.build_tables(
        [0, 3, 0, 0], [2, 4, 17, 1], table, [0, 1, 0, 0], [5, 6], 2, 26, 12, served)
    assert served == [2, 4, 0, 0] and q == [0, 2, 6, 6, 6] and counts == [1, 1, 0, 0] and left == 1
    assert list(slots[:6]) == [96, 97] + [9 * 16 + i for i in range(3, 7)] and set(slots[6:]) == {-1}
    assert list(pos[:6]) == [0, 1, 3, 4, 5, 6] and new == [0, 1, 1, 1, 1] and codes == {S.OUT_OF_PAGES}


def test_without_them_a_sequence_without_pages_is_committed():
    """The plain build packs all blocks: who takes its block lengths on moves the
    context of a sequence past tokens that are not in the cache."""
    ctx, T = [0, 0], [2, 2]
    served = []
    a = S.build_tables(ctx, T, np.full((2, 1), -1), [0, 0], [4], 1, 4, 8)
    S.build_tables(ctx, T, np.full((2, 1), -1), [0, 0], [4], 1, 4, 8, served)
    assert list(a[6]) == [64, 65, -1, -1] and served == [2, 0]
    x, y = np.array([1, 2, 3, 4]), np.array([2, 5, 4, 6])
    assert O.accept_commit(x, y, np.array(T), np.array(ctx))[1].tolist() == [2, 2]
    assert O.accept_commit(x, y, np.array(served), np.array(ctx))[1].tolist() == [2, 0]


SERVED = TABLES[:18] + ["served"] + TABLES[18:]
SERVED_OK = dict(TABLES_OK, served=F)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(n=-1), -1), (dict(P=32), -2), (dict(maxp=2 ** 27), -1),
    *[({k: None}, -1) for k in "ctx T tab cnt cnto free fc fco q new pos slots served".split()],
])
def test_argument_errors(lib, kw, code):  # noqa: F811
    assert call(lib.splash_build_tables_served, SERVED, SERVED_OK, kw) == code
