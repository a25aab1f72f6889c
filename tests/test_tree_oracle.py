"""The tree oracle on cases worked by hand, and against identities that its
definitions fix (CPU)."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import splash_oracle as O
from oracle import tree_oracle as T

#        0
#      1   2
#     3 4   5
#            6
PARENTS = [-1, 0, 0, 1, 1, 2, 5]


def test_masks_of_a_small_tree():
    m, d, pos, codes = T.tree_masks(PARENTS, [0, 7], [10], 1)
    assert [int(x) for x in m[:, 0]] == [0b1, 0b11, 0b101, 0b1011, 0b10011, 0b100101, 0b1100101]
    assert d.tolist() == [0, 1, 1, 2, 2, 2, 3] and pos.tolist() == [10, 11, 11, 12, 12, 12, 13]
    assert codes == set()


def test_a_chain_sees_what_a_block_sees():
    n = 40
    m, d, pos, _ = T.tree_masks([t - 1 for t in range(n)], [0, n], [3], 2)
    for t in range(n):
        assert T.seen_nodes(m[t], n).tolist() == [j <= t for j in range(n)]
    assert pos.tolist() == list(range(3, 3 + n))


def test_a_parent_out_of_range_is_none():
    m, d, _, codes = T.tree_masks([-1, 1, 0, 7], [0, 4], [0], 1)
    assert codes == {T.BAD_TREE} and m[:, 0].tolist() == [1, 2, 5, 8] and d.tolist() == [0, 0, 1, 0]


def test_the_accepted_path():
    tok = [9, 1, 2, 3, 4, 5, 6]
    #        target after each node
    for y, path, nxt in [([2, 0, 5, 0, 0, 6, 8], [0, 2, 5, 6], 8), ([1, 4, 0, 0, 7, 0, 0], [0, 1, 4], 7),
                         ([3, 4, 0, 0, 7, 0, 0], [0], 3), ([2, 0, 6, 0, 0, 6, 8], [0, 2], 6)]:
        acc, n, ctx, rows, toks, codes = T.accept_tree(tok, PARENTS, y, [0, 7], [20])
        assert acc == [len(path) - 1] and n == [nxt] and ctx == [20 + len(path)] and not codes
        assert rows.tolist() == path + [-1] * (7 - len(path))
        assert toks.tolist() == [tok[i] for i in path] + [-1] * (7 - len(path))


def test_of_equal_siblings_the_first_is_taken_and_a_chain_is_accept_commit():
    acc, nxt, _, rows, _, _ = T.accept_tree([5, 7, 7, 8], [-1, 0, 0, 2], [7, 1, 8, 2], [0, 4], [0])
    assert acc == [1] and nxt == [1] and rows.tolist() == [0, 1, -1, -1]
    rng = np.random.default_rng(0)
    for _ in range(50):
        lens = rng.integers(0, 6, 4)
        off = np.concatenate([[0], np.cumsum(lens)])
        x, y = rng.integers(0, 3, off[-1]), rng.integers(0, 3, off[-1])
        parents = [t - 1 for n in lens for t in range(n)]
        a, c, n = O.accept_commit(x, y, lens, [1, 2, 3, 4])
        got = T.accept_tree(x, parents, y, off, [1, 2, 3, 4])
        assert got[0] == a.tolist() and got[1] == n.tolist() and got[2] == c.tolist()


def test_nodes_without_a_token_and_other_roots_are_never_accepted():
    acc, nxt, *_ = T.accept_tree([5, -1, 4], [-1, 0, -1], [-1, 0, 0], [0, 3], [0])
    assert acc == [0] and nxt == [-1]
    acc, nxt, *_ = T.accept_tree([5, 4], [-1, -1], [4, 0], [0, 2], [0])
    assert acc == [0] and nxt == [4]


def test_compact_reads_before_it_writes():
    rows = np.arange(10) * 11
    # slots 4, 9, 2, 7, 0 of a tree of five; its path is nodes 0, 2, 3
    got = T.compact(rows, [4, 9, 2, 7, 0], [0, 2, 3, -1, -1], [0, 5], [2])
    want = rows.copy()
    want[9], want[2] = rows[2], rows[7]
    assert got.tolist() == want.tolist()


def test_logprobs_by_hand():
    z = np.array([[0.0, math.log(3), 0.0, -np.inf], [7, 7, 7, 7], [-np.inf] * 4,
                  [np.inf, 0, np.inf, 1], [np.nan, 2, 2, np.nan]])
    lp, ent, ids, tops = T.logprobs(z, [1, 2, 0, 0, 0], 3)
    assert lp[0] == pytest.approx(math.log(0.6)) and lp[1] == pytest.approx(-math.log(4))
    assert ent[0] == pytest.approx(-(0.6 * math.log(0.6) + 0.4 * math.log(0.2)))
    assert ent[1] == pytest.approx(math.log(4)) and lp[2] == -np.inf and ent[2] == 0
    assert ids[0].tolist() == [1, 0, 2] and ids[1].tolist() == [0, 1, 2]
    assert ids[2].tolist() == [-1] * 3 and tops[2].tolist() == [-np.inf] * 3
    assert ids[3].tolist() == [0, 2, 3] and lp[3] == pytest.approx(-math.log(2)) and tops[3, 2] < -1e30
    assert ids[4].tolist() == [1, 2, -1] and lp[4] == -np.inf and ent[4] == pytest.approx(math.log(2))


def _pool(rng, pages, hkv, D):
    pool = O.PagedPool(pages, hkv, 16, D)
    pool.k_codes[:] = rng.integers(-127, 128, pool.k_codes.shape)
    pool.v_codes[:] = rng.integers(-127, 128, pool.v_codes.shape)
    pool.k_scales[:] = rng.uniform(0.005, 0.02, pool.k_scales.shape)
    pool.v_scales[:] = rng.uniform(0.005, 0.02, pool.v_scales.shape)
    return pool


def test_attention_of_a_chain_is_verify_attention():
    rng = np.random.default_rng(1)
    pool, table = _pool(rng, 6, 2, 16), rng.permutation(6).reshape(2, 3)
    ctx, lens = [19, 0], [5, 7]
    q = rng.standard_normal((12, 4, 16))
    parents = [t - 1 for n in lens for t in range(n)]
    m, *_ = T.tree_masks(parents, [0, 5, 12], ctx, 1)
    o, lse, _ = T.attention(q, pool, table, ctx, lens, m, 2, 0.25)
    want, wl = O.attention(q, pool, table, np.array(ctx), np.array(lens), 2, 0.25)
    assert np.abs(o - want).max() < 1e-12 and np.abs(lse - wl).max() < 1e-12


def test_attention_of_a_node_is_that_of_its_path_alone():
    """The row of a node equals the last row of a chain that holds its path's keys."""
    rng = np.random.default_rng(2)
    pool, table = _pool(rng, 4, 1, 16), np.array([[2, 0, 3, 1]])
    ctx, n = 21, 7
    q = rng.standard_normal((n, 2, 16))
    m, *_ = T.tree_masks(PARENTS, [0, n], [ctx], 1)
    o, lse, _ = T.attention(q, pool, table, [ctx], [n], m, 1, 0.25)
    for t in range(n):
        path = T.ancestors(PARENTS, t)[::-1]
        k, v = O.gather_keys(pool, table[0], 0, ctx + n)
        keep = list(range(ctx)) + [ctx + j for j in path]
        want, wl = O.attention_seq_head(q[t:t + 1], k[keep], v[keep], len(keep) - 1, 0.25)
        assert np.abs(o[t] - want[0]).max() < 1e-12 and np.abs(lse[t] - wl[0]).max() < 1e-12


def test_a_row_that_sees_nothing_and_bits_past_the_tree():
    rng = np.random.default_rng(3)
    pool, table = _pool(rng, 2, 1, 16), np.array([[1, 0]])
    q = rng.standard_normal((3, 1, 16))
    m = np.array([[0], [0xfffffff8], [0b100]], np.uint32)
    o, lse, _ = T.attention(q, pool, table, [0], [3], m, 1, 0.25)
    assert not o[:2].any() and (lse[:2] == -np.inf).all()
    k, v = O.gather_keys(pool, table[0], 0, 3)
    assert np.abs(o[2, 0] - v[2]).max() < 1e-12          # one key
