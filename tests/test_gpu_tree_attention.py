"""Attention over a tree of drafts on the GPU against the fp64 oracle.

Bounds, per row. A score is off by at most d = (2 (D + 8) 2^-24) qk, where qk =
sm_scale * sum_d |q_d k_d| of the key with the largest sum: the products of the codes
and the rescaled q are exact, their D additions and the scale are fp32 (twice a half
step, for an accumulator that cuts instead of rounding); the exponent's argument and
ex2 add 2^-21. So weights are off by r = 2 (d + 2^-21) of themselves, and

  lse: d + 2^-21 + 2^-22 |lse| + 2^-21 (the sums and the logarithm)
  out: 2^-8 |o| (bf16, half a step) + (r + 2^-11) sum_j p_j |v_j| (each p_j s_V,j is
       rounded to fp16 once, half a step 2^-11 at most) + n 127 2^-25 / S (where that
       product is a subnormal fp16: half a step 2^-25 times a code; S = sum_j exp(s_j -
       max) is not above the kernel's sum, whose reference is a key's score).
"""
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

from oracle import splash_oracle as O  # noqa: E402
from oracle import tree_oracle as T  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402


def i32(a):
    a = np.ascontiguousarray(a)
    return torch.tensor(a.astype(np.int64) if a.dtype == np.uint32 else a,
                        device="cuda").to(torch.int64).to(torch.int32)


class Case:
    """A poisoned pool, a tree per sequence and everything a call takes."""

    def __init__(self, seed, ctx, lens, hq, hkv, D, kind="tree", words=None, unit=0.01):
        rng = np.random.default_rng(seed)
        self.ctx, self.lens, self.hq, self.hkv, self.D = ctx, lens, hq, hkv, D
        n = self.n = int(sum(lens))
        self.most = max(lens)
        self.words = words or -(-self.most // 32)
        held = [-(-(c + t) // 16) for c, t in zip(ctx, lens)]
        pages = self.pages = sum(held) + 3
        perm = rng.permutation(pages)
        self.table = np.full((len(ctx), max(held) + 1), -1, np.int64)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = perm[at:at + h]
            at += h
        self.codes = np.full((pages, hkv, 2, 16, D), 127, np.int8)
        self.scales = np.full((2, pages, hkv, 16), np.inf, np.float32)
        self.scales[1] = np.nan
        for b in range(len(ctx)):
            for j in range(ctx[b] + lens[b]):
                pg, s = self.table[b, j // 16], j % 16
                self.codes[pg, :, :, s] = rng.integers(-127, 128, (hkv, 2, D))
                self.scales[:, pg, :, s] = unit * rng.uniform(0.5, 1.0, (2, hkv))
        self.pool = O.PagedPool(pages, hkv, 16, D)
        self.pool.k_codes, self.pool.v_codes = self.codes[:, :, 0], self.codes[:, :, 1]
        self.pool.k_scales, self.pool.v_scales = self.scales[0], self.scales[1]
        self.masks = np.zeros((n, self.words), np.uint32)
        off = self.off = np.concatenate([[0], np.cumsum(lens)])
        for b, t in enumerate(lens):
            lo, hi = off[b], off[b + 1]
            if kind == "random":                       # any bits, past the tree too
                self.masks[lo:hi] = rng.integers(0, 2 ** 32, (t, self.words), dtype=np.uint32)
            elif kind == "full":
                self.masks[lo:hi] = 0xffffffff
            elif kind == "sparse":                     # a third of the rows sees no node
                m = rng.integers(0, 2 ** 32, (t, self.words), dtype=np.uint32) & \
                    rng.integers(0, 2 ** 32, (t, self.words), dtype=np.uint32)
                m[rng.random(t) < 0.34] = 0
                self.masks[lo:hi] = m
            elif kind != "empty":
                back = 1 if kind == "chain" else 6
                parents = [t - 1 - int(rng.integers(0, min(back, t))) if t else -1 for t in range(t)]
                self.masks[lo:hi] = T.tree_masks(parents, [0, t], [0], self.words)[0]
        self.q = torch.tensor(rng.standard_normal((n, hq, D)), dtype=torch.bfloat16, device="cuda")
        codes = torch.tensor(self.codes, device="cuda")
        self.dev = (codes[:, :, 0], codes[:, :, 1], torch.tensor(self.scales[0], device="cuda"),
                    torch.tensor(self.scales[1], device="cuda"))
        self.sm = D ** -0.5

    def run(self, ctas=0, status=None, extra=0, stream=None, **over):
        n = self.n + extra                             # rows behind the last sequence
        q = torch.cat([self.q, self.q.new_full((extra, self.hq, self.D), 7)])
        masks = torch.cat([i32(self.masks), i32(np.full((extra, self.words), -1))])
        out = torch.full((n, self.hq, self.D), -3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, self.hq), -3.0, device="cuda")
        a = dict(page_table=i32(self.table), context_lens=i32(self.ctx), block_lens=i32(self.lens),
                 max_block_len=self.most)
        a.update(over)
        ws = sk.alloc_tree_workspace(len(self.ctx), n, self.hq, self.hkv, self.D,
                                     a["max_block_len"], ctas=ctas)
        ws.fill_(0xa5)
        sk.splash_verify_attention_tree(q, *self.dev, tree_masks=masks, sm_scale=self.sm, out=out,
                                        lse=lse, workspace=ws, device_status=status, ctas=ctas,
                                        stream=stream, **a)
        return out, lse

    def check(self, out, lse, rows=slice(None)):
        want, wl, (av, qk, total) = T.attention(self.q.double().cpu().numpy(), self.pool,
                                                self.table, self.ctx, self.lens, self.masks,
                                                self.hkv, self.sm)
        o, got = out[:self.n].double().cpu().numpy()[rows], lse[:self.n].double().cpu().numpy()[rows]
        want, wl, av, qk, total = want[rows], wl[rows], av[rows], qk[rows], total[rows]
        keys = max(c + t for c, t in zip(self.ctx, self.lens))
        d = 2 * (self.D + 8) * 2.0 ** -24 * qk + 2.0 ** -21
        none = np.isneginf(wl)
        assert np.array_equal(np.isneginf(got), none) and not o[none].any()
        live = ~none
        off = np.abs(got[live] - wl[live])
        assert (off <= (d + 2.0 ** -21)[live] + 2.0 ** -22 * np.abs(wl[live])).all(), off.max()
        bound = 2.0 ** -8 * np.abs(want) + (2 * d[..., None] + 2.0 ** -11) * av \
            + (keys * 127 * 2.0 ** -25 / total)[..., None]
        err = np.abs(o - want)
        assert (err <= bound)[live].all(), (err / np.maximum(bound, 1e-30))[live].max()


SHAPES = [  # contexts, nodes, query heads, KV heads, head dimension
    ([0], [1], 1, 1, 64), ([0], [1], 4, 2, 256), ([1], [3], 6, 1, 128),
    ([63, 0, 17, 64], [5, 4, 0, 16], 8, 2, 128), ([130, 65], [33, 1], 4, 4, 64),
    ([15, 16, 500], [32, 31, 2], 14, 2, 64), ([200, 3], [21, 64], 12, 2, 256),
    ([40, 100], [65, 7], 8, 2, 128), ([70], [128], 6, 2, 64), ([10, 0], [256, 100], 2, 1, 128),
    ([300], [97], 8, 1, 64), ([1000, 1, 90], [16, 1, 9], 24, 4, 256),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
@pytest.mark.parametrize("kind", ["tree", "sparse"])
def test_matches_the_oracle(shape, kind):
    c = Case(len(str(shape)), *shape, kind=kind)
    status = i32([0])
    out, lse = c.run(status=status, extra=3)
    assert status.item() == 0
    c.check(out, lse)
    assert (out[c.n:] == -3).all() and (lse[c.n:] == -3).all()


@pytest.mark.parametrize("kind", ["random", "full", "empty", "chain"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctas", [0, 1, 3, 211])
def test_masks_of_any_kind_and_any_split(kind, D, ctas):
    c = Case(D + ctas, [37, 0, 250], [70, 66, 40], 4, 2, D, kind=kind, words=4)
    c.check(*c.run(ctas=ctas))


def test_a_chain_is_verify_attention():
    for D in (64, 128, 256):
        c = Case(D, [37, 400, 0], [9, 16, 3], 8, 2, D, kind="chain")
        out, lse = c.run()
        c.check(out, lse)
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        ws = sk.alloc_workspace(3, c.n, 8, 2, D, 16)
        sk.splash_verify_attention(c.q, *c.dev, i32(c.table), i32(c.ctx), i32(c.lens), c.sm, 16, o2,
                                   l2, ws)
        c.check(o2, l2)                    # the same bounds hold for both


def test_the_same_call_is_bitwise_the_same_and_page_numbers_do_not_matter():
    c = Case(5, [300, 20], [50, 9], 8, 2, 128)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    perm = np.random.default_rng(0).permutation(c.pages)
    back = np.argsort(perm)
    d = Case(5, [300, 20], [50, 9], 8, 2, 128)
    codes = torch.tensor(c.codes[back], device="cuda")
    d.dev = (codes[:, :, 0], codes[:, :, 1], torch.tensor(c.scales[0][back], device="cuda"),
             torch.tensor(c.scales[1][back], device="cuda"))
    d.table = np.where(c.table >= 0, perm[c.table], -1)
    e = d.run()
    assert torch.equal(a[0], e[0]) and torch.equal(a[1], e[1])


@pytest.mark.parametrize("unit", [1e-5, 10.0])
def test_scales_far_from_one(unit):
    c = Case(8, [90], [20], 4, 1, 128, unit=1.0)
    c.scales[0] *= 0.01
    c.scales[1] *= unit
    c.dev = (*c.dev[:2], torch.tensor(c.scales[0], device="cuda"),
             torch.tensor(c.scales[1], device="cuda"))
    c.check(*c.run())


def test_sharp_rows_and_zero_queries():
    """Scores of hundreds (one key takes all), of zero (all alike)."""
    c = Case(9, [500], [24], 4, 2, 128)
    c.q[::2] *= 40
    c.q[1::4] = 0
    c.check(*c.run())


def test_bad_lengths_and_pages_leave_the_others():
    c = Case(11, [40, 60, 33], [7, 9, 5], 4, 2, 128)
    keep = np.r_[0:7, 16:21]
    for over in (dict(context_lens=i32([40, -1, 33])), dict(context_lens=i32([40, 10 ** 6, 33]))):
        status = i32([0])
        out, lse = c.run(status=status, **over)
        assert status.item() == sk.DEVICE_BAD_LENGTH
        c.check(out, lse, keep)
        assert (out[7:16] == -3).all() and (lse[7:16] == -3).all()
    # more rows than the caller has: nothing is written
    status = i32([0])
    out, lse = c.run(status=status, block_lens=i32([7, 9, 6]))
    assert status.item() == sk.DEVICE_BAD_LENGTH and (out == -3).all() and (lse == -3).all()
    # a tree above the stated bound
    status = i32([0])
    out, lse = c.run(status=status, max_block_len=8)
    assert status.item() == sk.DEVICE_BAD_LENGTH
    c.check(out, lse, keep)
    # a page id where a page is needed
    for bad in (-1, c.pages, 2 ** 31 - 1):
        t = c.table.copy()
        t[1, 1] = bad
        status = i32([0])
        out, lse = c.run(status=status, page_table=i32(t))
        assert status.item() == sk.DEVICE_BAD_PAGE
        c.check(out, lse, keep)


def test_many_sequences_on_both_sides_of_the_plan_sizes():
    for B in (128, 129, 1024, 1025):
        rng = np.random.default_rng(B)
        ctx, lens = rng.integers(0, 40, B).tolist(), rng.integers(0, 4, B).tolist()
        lens[0] = 3
        c = Case(B, ctx, lens, 2, 1, 64)
        c.check(*c.run())


def test_on_another_stream_and_in_a_graph():
    c = Case(13, [100, 7], [40, 12], 8, 2, 128)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run()
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    ctx, lens, table = i32(c.ctx), i32(c.lens), i32(c.table)
    masks, q = i32(c.masks), c.q.clone()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = sk.alloc_tree_workspace(2, c.n, 8, 2, 128, 40)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.splash_verify_attention_tree(q, *c.dev, table, ctx, lens, masks, c.sm, 40, out, lse, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(want[0], out) and torch.equal(want[1], lse)
    # other lengths of the same batch, the same graph
    d = Case(13, [100, 7], [40, 12], 8, 2, 128)
    d.ctx, d.lens = [90, 2], [40, 12]
    ctx.copy_(i32(d.ctx))
    g.replay()
    torch.cuda.synchronize()
    d.check(out, lse)


def test_a_long_cache_past_four_gigabytes():
    """The codes of the last pages lie past 32 bits of offset."""
    D, hkv = 256, 4
    pages = 2 ** 32 // (hkv * 2 * 16 * D) + 40
    codes = torch.zeros((pages, hkv, 2, 16, D), dtype=torch.int8, device="cuda")
    ks = torch.full((pages, hkv, 16), float("nan"), device="cuda")
    vs = torch.full((pages, hkv, 16), float("nan"), device="cuda")
    c = Case(17, [70], [5], 8, hkv, D)
    for j, pg in enumerate(c.table[0, :5]):
        codes[pages - 1 - j] = torch.tensor(c.codes[pg], device="cuda")
        ks[pages - 1 - j] = torch.tensor(c.scales[0][pg], device="cuda")
        vs[pages - 1 - j] = torch.tensor(c.scales[1][pg], device="cuda")
    want = c.run()
    c.dev = (codes[:, :, 0], codes[:, :, 1], ks, vs)
    got = c.run(page_table=i32([[pages - 1, pages - 2, pages - 3, pages - 4, pages - 5, -1]]))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
