"""Page tables, slot maps and released pages on the GPU against the step oracle
(integers: equality)."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from speculative_verify_attention_kv_gb300 import build as _build  # noqa: E402

if not os.path.exists(_build.LIB):
    _build.build()

from oracle import step_oracle as S  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def scene(seed, B, ctx_hi, T_of, extra_held=0.3, max_pages=None):
    """Lengths, a table whose held entries are distinct pages, and a free list."""
    r = np.random.default_rng(seed)
    ctx = r.integers(0, ctx_hi + 1, B)
    T = np.array([T_of(r) for _ in range(B)])
    held = [S.pages_of(int(c)) + int(r.random() < extra_held) for c in ctx]
    mp = max_pages or max([S.pages_of(int(c + max(t, 0))) + 1 for c, t in zip(ctx, T)] + [1])
    held = [min(h, mp) for h in held]
    total = sum(held) + sum(S.pages_of(int(c + max(t, 0))) for c, t in zip(ctx, T)) + 3
    perm = r.permutation(total)
    table = np.full((B, mp), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    return ctx, T, table, np.array(held, np.int64), perm[at:], total


def build(ctx, T, table, counts, free, free_count, n, num_pages, in_place=False, cap=None):
    B = len(ctx)
    t = i32(table)
    c, fc = i32(counts), i32([free_count])
    co, fo = (c, fc) if in_place else (torch.full_like(c, -9), torch.full_like(fc, -9))
    f = i32(free if cap is None else free[:cap])
    q, new = (torch.full((B + 1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pos, slots = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.splash_build_tables(i32(ctx), i32(T), t, c, f, fc, q, new, pos, slots, num_pages,
                           page_counts_out=None if in_place else co,
                           free_count_out=None if in_place else fo, device_status=st)
    torch.cuda.synchronize()
    if not in_place:
        assert c.tolist() == list(counts) and fc.item() == free_count
    return (t, co, fo, q, new, pos, slots, st), f


def check(got, want):
    t, counts, left, q, new, pos, slots, codes = want
    assert np.array_equal(got[0].cpu().numpy(), t)
    assert got[1].tolist() == counts and got[2].item() == left
    assert got[3].tolist() == q and got[4].tolist() == new
    assert np.array_equal(got[5].cpu().numpy(), pos)
    assert np.array_equal(got[6].cpu().numpy(), slots)
    assert got[7].item() in codes if codes else got[7].item() == 0


CASES = [
    # (B, longest context, block lengths): one CTA, the scan's chunk edges, the
    # second kernel (over 4096 tokens), offsets kept out of shared memory
    (1, 0, [1]), (1, 15, [1]), (1, 16, [0]), (3, 100, [0, 1, 17]), (64, 2000, [1, 4, 8, 16]),
    (128, 300, [0, 5]), (129, 300, [0, 5]), (1024, 64, [1, 2]), (1025, 64, [1, 3]),
    (2500, 40, [0, 1, 4]), (3, 50, [4096]), (5, 7000, [1000, 1, 3333]), (2, 0, [40000, 25001]),
    (300, 500, [16, 40]),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pad", [0, 7])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_build_matches_the_oracle(case, pad, in_place):
    B, hi, lens = case
    ctx, T, table, counts, free, total = scene(B + hi, B, hi, lambda r: int(r.choice(lens)))
    n = int(T.sum()) + pad
    want = S.build_tables(ctx, T, table, counts, free, len(free), n, total)
    got, _ = build(ctx, T, table, counts, free, len(free), n, total, in_place)
    check(got, want)


@pytest.mark.parametrize("B,seed", [(6, 1), (200, 2), (1500, 3)])
def test_a_short_free_list_serves_in_order(B, seed):
    ctx, T, table, counts, free, total = scene(seed, B, 200, lambda r: int(r.choice([0, 1, 9, 40])))
    n = int(T.sum())
    full = S.build_tables(ctx, T, table, counts, free, len(free), n, total)
    need = len(free) - full[2]
    for have in (0, 1, need // 2, need - 1, need):
        want = S.build_tables(ctx, T, table, counts, free[:have], have, n, total)
        got, _ = build(ctx, T, table, counts, free, have, n, total)
        check(got, want)
    # a count past the list is cut to it
    want = S.build_tables(ctx, T, table, counts, free[:2], 99, n, total)
    got, _ = build(ctx, T, table, counts, free, 99, n, total, cap=2)
    check(got, want)


def test_bad_lengths_and_pages_leave_the_others():
    ctx, T, table, counts, free, total = scene(5, 9, 100, lambda r: 5, max_pages=9)
    ctx[1], T[2], ctx[3], counts[4] = -1, -4, 9 * 16, 77
    table[5, 0] = total                              # out of the pool
    table[6, 0] = -1
    ctx[5], ctx[6] = 3, 2                            # blocks inside those pages
    counts[5] = max(counts[5], 1)
    counts[6] = max(counts[6], 1)
    n = int(np.maximum(T, 0).sum())
    want = S.build_tables(ctx, T, table, counts, free, len(free), n, total)
    assert want[-1] == {S.BAD_LENGTH, S.BAD_PAGE}
    check(build(ctx, T, table, counts, free, len(free), n, total)[0], want)
    # rows past the caller's count: the last sequences get nothing
    want = S.build_tables(ctx, T, table, counts, free, len(free), n - 12, total)
    check(build(ctx, T, table, counts, free, len(free), n - 12, total)[0], want)
    # a page that the free list should not hold
    bad = np.array(free)
    bad[-1] = -5
    want = S.build_tables([0], [3], [[-1]], [0], bad, len(bad), 3, total)
    check(build([0], [3], [[-1]], [0], bad, len(bad), 3, total)[0], want)


def test_huge_block_lengths_do_not_overflow():
    big = 2 ** 31 - 1
    T = [big, big, 3]
    want = S.build_tables([0, 5, 0], T, np.full((3, 4), -1), [0, 0, 0], [1, 2], 2, 10, 8)
    got, _ = build([0, 5, 0], T, np.full((3, 4), -1), [0, 0, 0], [1, 2], 2, 10, 8)
    assert got[3].tolist() == [0, big, big, big]     # held at the largest 32-bit offset
    assert got[1].tolist() == want[1] and set(got[6].tolist()) == {-1}
    assert got[7].item() == S.BAD_LENGTH


def test_empty_batch():
    got, _ = build([], [], np.zeros((0, 4)), [], [3, 4], 2, 5, 8)
    assert got[2].item() == 2 and got[3].tolist() == [0] and set(got[6].tolist()) == {-1}


@pytest.mark.parametrize("B,hi", [(1, 0), (1, 40), (7, 100), (64, 3000), (130, 900), (2300, 60)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_matches_the_oracle(B, hi, in_place):
    ctx, T, table, counts, free, total = scene(B * 7 + hi, B, hi, lambda r: 1)
    r = np.random.default_rng(B)
    keep = np.array([r.choice([0, -1, int(c), max(0, int(c) - 20), int(c) + 999]) for c in ctx])
    n0 = len(free)
    for cap in (total, n0 + 3, n0):
        stack = np.full(cap, -7)
        stack[:n0] = free
        want = S.release_pages(keep, table, counts, stack, n0)
        c, fc, f = i32(counts), i32([n0]), i32(stack)
        co, fo = (c, fc) if in_place else (torch.full_like(c, -9), torch.full_like(fc, -9))
        off = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sk.splash_release_pages(i32(keep), i32(table), c, f, fc, off,
                                page_counts_out=None if in_place else co,
                                free_count_out=None if in_place else fo, device_status=st)
        torch.cuda.synchronize()
        assert co.tolist() == want[0] and f.tolist() == want[1] and fo.item() == want[2]
        assert off.tolist() == want[3]
        assert st.item() == (S.BAD_LENGTH if want[4] else 0)


def test_pages_go_round_and_none_is_lost():
    """Steps of growth, trimming and turnover: no page is ever held twice, and
    free and held pages are always all of them."""
    B, total, mp = 24, 400, 40
    r = np.random.default_rng(9)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    counts = torch.zeros(B, dtype=torch.int32, device="cuda")
    free, fc = i32(r.permutation(total)), i32([total])
    ctx = np.zeros(B, np.int64)
    q, new, off = (torch.zeros(B + 1, dtype=torch.int32, device="cuda") for _ in range(3))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(30):
        T = r.integers(0, 20, B)
        n = int(T.sum())
        pos, slots = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
        sk.splash_build_tables(i32(ctx), i32(T), table, counts, free, fc, q, new, pos, slots, total,
                               device_status=st)
        assert st.item() == 0 and len(set(slots.tolist())) == n
        ctx = ctx + np.minimum(T, r.integers(0, 20, B))          # what was accepted
        done = r.random(B) < 0.1
        ctx[done | (ctx > 16 * mp - 40)] = 0
        sk.splash_release_pages(i32(ctx), table, counts, free, fc, off, device_status=st)
        c, t = counts.tolist(), table.cpu().numpy()
        held = [int(p) for b in range(B) for p in t[b, :c[b]]]
        assert c == [S.pages_of(int(x)) for x in ctx]
        assert sorted(held + free.tolist()[:fc.item()]) == list(range(total))
    assert st.item() == 0


def test_a_captured_call_follows_its_inputs():
    ctx, T, table, counts, free, total = scene(11, 40, 400, lambda r: 200)
    n = int(T.sum())
    d = dict(ctx=i32(ctx), T=i32(T), table=i32(table), counts=i32(counts), free=i32(free),
             fc=i32([len(free)]))
    co, fo = torch.empty_like(d["counts"]), torch.empty_like(d["fc"])
    q, new = (torch.empty(41, dtype=torch.int32, device="cuda") for _ in range(2))
    pos, slots = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))

    def call():
        sk.splash_build_tables(d["ctx"], d["T"], d["table"], d["counts"], d["free"], d["fc"], q, new,
                               pos, slots, total, page_counts_out=co, free_count_out=fo)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for T2 in (200, 33, 1):
        T = np.full(40, T2)
        d["T"].copy_(i32(T))
        d["table"].copy_(i32(table))
        g.replay()
        torch.cuda.synchronize()
        want = S.build_tables(ctx, T, table, counts, free, len(free), n, total)
        assert np.array_equal(slots.cpu().numpy(), want[6]) and co.tolist() == want[1]
        assert np.array_equal(d["table"].cpu().numpy(), want[0]) and fo.item() == want[2]


def test_misaligned_outputs():
    """positions and slots as views that start off a 16-byte boundary."""
    ctx, T, table, counts, free, total = scene(3, 5, 90, lambda r: 7)
    n = int(T.sum())
    want = S.build_tables(ctx, T, table, counts, free, len(free), n, total)
    big = torch.full((2, n + 3), -9, dtype=torch.int32, device="cuda")
    flat = big.reshape(-1)
    pos, slots = flat[1:1 + n], flat[n + 3:2 * n + 3]
    q, new = (torch.empty(6, dtype=torch.int32, device="cuda") for _ in range(2))
    sk.splash_build_tables(i32(ctx), i32(T), i32(table), i32(counts), i32(free), i32([len(free)]), q,
                           new, pos, slots, total)
    torch.cuda.synchronize()
    assert np.array_equal(pos.cpu().numpy(), want[5]) and np.array_equal(slots.cpu().numpy(), want[6])
    assert flat[0].item() == -9 and set(flat[n + 1:n + 3].tolist()) == {-9}


@pytest.mark.parametrize("ctx0", [0, 1, 15, 16, 37])
def test_bad_pages_inside_long_blocks(ctx0):
    """Blocks of thousands of rows from any offset in a page, held pages and pages
    of the free list out of the pool among theirs."""
    ctx, T = np.array([ctx0, 5, ctx0 + 3]), np.array([3001, 1, 5200])
    held = np.array([120, 1, 200])
    total, width = 900, 400
    r = np.random.default_rng(ctx0)
    ids = r.permutation(total)
    table = np.full((3, width), -1)
    at = 0
    for b in range(3):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = ids[at:].copy()
    table[0, 7], table[2, 199], table[2, 0] = total, -3, total + 5
    free[-9], free[-40] = -1, total
    n = int(T.sum()) + 5
    want = S.build_tables(ctx, T, table, held, free, len(free), n, total)
    assert want[-1] == {S.BAD_PAGE}
    check(build(ctx, T, table, held, free, len(free), n, total)[0], want)
