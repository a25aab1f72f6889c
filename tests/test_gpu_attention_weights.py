"""Attention where one key holds most of the weight and its own value is small, so that the
output is what the others add: trees and chains, against the fp64 oracle.

Bounds as in test_gpu_tree_attention.py but for the products p s_V that are rounded to
fp16: they carry a power of two f that puts the largest V scale of the keys that a row
sees, M, at 2^5 <= f M < 2^7. So a subnormal product is off by 2^-25 / f <= M 2^-30, times a
code of at most 127, for n keys: n 127 M 2^-30 / S.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from oracle import splash_oracle as O  # noqa: E402
from oracle import tree_oracle as T  # noqa: E402

from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

from test_gpu_tree_attention import Case, i32  # noqa: E402


class Sink(Case):
    """Key `at` of every sequence has a score about `gap` above the others' (in e^: so many
    times their weight) and a value `small` times theirs; V scales `unit` times 0.5 to 1,
    and `growth` times that from key `grows` on."""

    def __init__(self, seed, ctx, lens, hq, hkv, D, gap, at=0, small=0.0, unit=0.01, grows=None,
                 growth=1.0, kind="tree"):
        super().__init__(seed, ctx, lens, hq, hkv, D, kind=kind)
        rng = np.random.default_rng(seed + 1)
        u = rng.choice([-1.0, 1.0], (hkv, D))
        q = 0.5 * np.repeat(u, hq // hkv, 0)[None] + 0.05 * rng.standard_normal((self.n, hq, D))
        self.q = torch.tensor(q, dtype=torch.bfloat16, device="cuda")
        self.scales[0] *= 0.01                          # the others' scores: next to nothing
        for b in range(len(ctx)):
            for j in range(ctx[b] + lens[b]):
                pg, s = self.table[b, j // 16], j % 16
                self.scales[1, pg, :, s] *= unit / 0.01 * (growth if grows and j >= grows else 1)
            pg, s = self.table[b, at // 16], at % 16
            self.codes[pg, :, 0, s] = (100 * u).astype(np.int8)
            self.scales[0, pg, :, s] = gap / (self.sm * 100 * 0.5 * D)
            self.scales[1, pg, :, s] = unit * small
        codes = torch.tensor(self.codes, device="cuda")
        self.pool.k_codes, self.pool.v_codes = self.codes[:, :, 0], self.codes[:, :, 1]
        self.pool.k_scales, self.pool.v_scales = self.scales[0], self.scales[1]
        self.dev = (codes[:, :, 0], codes[:, :, 1], torch.tensor(self.scales[0], device="cuda"),
                    torch.tensor(self.scales[1], device="cuda"))
        self.want, self.big = None, unit * max(1.0, growth) > 1e20

    def check(self, out, lse, rows=slice(None)):
        if self.want is None:
            # (poisoned scales are read as what they are: rows that see them are not looked at)
            self.want = T.attention(self.q.double().cpu().numpy(), self.pool, self.table, self.ctx,
                                    self.lens, self.masks, self.hkv, self.sm)
        want, wl, (av, qk, total) = self.want
        o, got = out[:self.n].double().cpu().numpy(), lse[:self.n].double().cpu().numpy()
        keys = max(c + t for c, t in zip(self.ctx, self.lens))
        M = max(m for b in range(len(self.ctx)) for j in range(self.ctx[b] + self.lens[b])
                for m in self.scales[1, self.table[b, j // 16], :, j % 16] if m < 1e29 or self.big)
        d = 2 * (self.D + 8) * 2.0 ** -24 * qk + 2.0 ** -21
        live = ~np.isneginf(wl)
        live[[r for r in range(self.n) if r not in np.arange(self.n)[rows]]] = False
        none = np.isneginf(wl)[rows]
        assert np.array_equal(np.isneginf(got)[rows], none) and not o[rows][none].any()
        off = np.abs(got - wl)[live]
        assert (off <= (d + 2.0 ** -21)[live] + 2.0 ** -22 * np.abs(wl[live])).all(), off.max()
        bound = 2.0 ** -8 * np.abs(want) + (2 * d[..., None] + 2.0 ** -11) * av \
            + (keys * 127 * M * 2.0 ** -30 / total)[..., None]
        err = np.abs(o - want)
        assert (err <= bound)[live].all(), (err / np.maximum(bound, 1e-30))[live].max()

    def chain(self, **more):
        o, lse = torch.empty_like(self.q), torch.empty((self.n, self.hq), device="cuda")
        ws = sk.alloc_workspace(len(self.ctx), self.n, self.hq, self.hkv, self.D, self.most,
                                ctas_per_class=more.get("ctas_per_class", 0),
                                shared="shared_lens" in more)
        status = i32([0])
        sk.splash_verify_attention(self.q, *self.dev, i32(self.table), i32(self.ctx),
                                   i32(self.lens), self.sm, self.most, o, lse, ws,
                                   device_status=status, path=sk.PATH_TENSOR, **more)
        assert status.item() == 0
        return o, lse

    def windowed(self, W):
        """What T.attention returns, where a row sees the last W keys up to its own."""
        q = self.q.double().cpu().numpy()
        sm, G = float(np.float32(self.sm)), self.hq // self.hkv
        out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
        av, qk, total = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
        row = 0
        for b, (c, n) in enumerate(zip(self.ctx, self.lens)):
            for h in range(self.hkv):
                k, v = O.gather_keys(self.pool, self.table[b], h, c + n)
                for t in range(n):
                    seen = slice(max(0, c + t - W + 1), c + t + 1)
                    for g in range(h * G, (h + 1) * G):
                        x = sm * (k[seen] @ q[row + t, g])
                        p = np.exp(x - x.max())
                        total[row + t, g] = p.sum()
                        lse[row + t, g] = x.max() + np.log(p.sum())
                        out[row + t, g] = p @ v[seen] / p.sum()
                        av[row + t, g] = p @ np.abs(v[seen]) / p.sum()
                        qk[row + t, g] = sm * (np.abs(k[seen]) @ np.abs(q[row + t, g])).max()
            row += n
        self.want = out, lse, (av, qk, total)
        return self


GAPS = [6.0, 9.0, 12.0, 16.0]                 # the sink's weight: 0.2 to 0.9999 of a row's


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("at", [0, 1500])
def test_trees_keep_small_weights(D, gap, at):
    c = Sink(41, [2000, 1700], [9, 40], 4, 2, D, gap, at, small=0.02)
    for ctas in (1, 3, 0):
        c.check(*c.run(ctas=ctas))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("unit", [1e-6, 1e-3, 1.0, 1e3, 1e6, 1e30])
def test_trees_at_any_size_of_the_values(D, unit):
    c = Sink(42, [700], [20], 4, 1, D, 9.0, small=0.02, unit=unit)
    for ctas in (1, 0):
        c.check(*c.run(ctas=ctas))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("growth", [3.0, 300.0, 1e7, 1e-4])
@pytest.mark.parametrize("grows", [33, 200, 701])
def test_trees_whose_values_grow_along_the_keys(D, growth, grows):
    """From inside the first tile, the context's middle and the tree's nodes on."""
    c = Sink(43, [700], [20], 4, 1, D, 9.0, small=0.02, grows=grows, growth=growth, kind="sparse")
    for ctas in (1, 2):
        c.check(*c.run(ctas=ctas))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("poison", [float("inf"), float("nan"), 1e30])
def test_the_values_of_masked_nodes_do_not_matter(D, poison):
    """A node that only itself sees, with scales of any value: the other rows as if it were
    not there."""
    c = Sink(44, [90], [24], 4, 1, D, 9.0, small=0.02)
    c.masks &= np.uint32(~(1 << 13) & 0xffffffff)
    c.masks[13] |= np.uint32(1 << 13)
    want = c.run(ctas=1)
    c.check(*want)
    rest = [r for r in range(24) if r != 13]
    pg, s = c.table[0, 103 // 16], 103 % 16
    for t in c.dev[2:]:
        t[pg, :, s] = poison
    got = c.run(ctas=1)
    for a, b in zip(want, got):
        assert torch.equal(a[rest], b[rest])


@pytest.mark.parametrize("poison", [float("inf"), 1e30])
def test_a_row_with_scales_of_its_own_does_not_hide_the_others(poison):
    """One node that only itself sees with a scale of any value, in the first tile, then one
    large value after another in the second."""
    c = Sink(46, [32], [96], 1, 1, 64, 9.0, small=0.02, kind="full")
    c.masks[:, 0] &= np.uint32(0xffffffff ^ (1 << 13))
    c.masks[13] = 0
    c.masks[13, 0] = 1 << 13
    rest = [r for r in range(96) if r != 13]
    c.scales[1, c.table[0, 45 // 16], :, 45 % 16] = poison
    for j in range(64, 128):
        at = (1, c.table[0, j // 16], slice(None), j % 16)
        was = c.scales[at].copy()
        c.scales[at] = 1e7
        c.dev = (*c.dev[:3], torch.tensor(c.scales[1], device="cuda"))
        c.want = None
        with np.errstate(all="ignore"):
            c.check(*c.run(ctas=1), rows=rest)
        c.scales[at] = was


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_same_call_again_and_the_same_bits(D):
    c = Sink(45, [3000, 40], [30, 64], 8, 2, D, 9.0, small=0.02, grows=900, growth=50.0)
    want = c.run()
    for _ in range(20):
        got = c.run()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("at", [0, 1500])
def test_chains_keep_small_weights(D, gap, at):
    c = Sink(51, [2000, 1700], [9, 16], 4, 2, D, gap, at, small=0.02, kind="chain")
    for ctas in (1, 3, 0):
        c.check(*c.chain(ctas_per_class=ctas))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("unit", [1e-6, 1e-3, 1.0, 1e3, 1e6, 1e30])
def test_chains_at_any_size_of_the_values(D, unit):
    c = Sink(52, [700], [16], 4, 1, D, 9.0, small=0.02, unit=unit, kind="chain")
    for ctas in (1, 0):
        c.check(*c.chain(ctas_per_class=ctas))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("growth", [3.0, 300.0, 1e7, 1e-4])
@pytest.mark.parametrize("grows", [33, 200, 701])
def test_chains_whose_values_grow_along_the_keys(D, growth, grows):
    c = Sink(53, [700], [20], 4, 1, D, 9.0, small=0.02, grows=grows, growth=growth, kind="chain")
    for ctas in (1, 2):
        c.check(*c.chain(ctas_per_class=ctas))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("W", [1, 40, 300, 5000])
@pytest.mark.parametrize("growth", [1.0, 1e5])
def test_windows_keep_small_weights(D, W, growth):
    c = Sink(54, [700, 30], [20, 9], 4, 1, D, 9.0, 640 if W == 300 else 0, small=0.02, grows=650,
             growth=growth, kind="chain") if W > 1 else \
        Sink(54, [700, 30], [20, 9], 4, 1, D, 9.0, 0, small=0.02, kind="chain")
    c.windowed(W)
    for ctas in (1, 3, 0):
        c.check(*c.chain(ctas_per_class=ctas, window=W))


@pytest.mark.parametrize("D", [128, 256])
def test_shared_prefixes_keep_small_weights(D):
    c = Sink(55, [1200, 1300, 1210], [5, 4, 3], 4, 2, D, 9.0, small=0.02, grows=1100, growth=40.0,
             kind="chain")
    c.table[1:, :64] = c.table[0, :64]               # the first 1024 keys
    c.check(*c.chain(shared_lens=i32([0, 1024, 1024])))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("poison", [float("inf"), float("nan"), 1e30])
def test_the_values_of_later_tokens_do_not_matter(D, poison):
    c = Sink(56, [110], [24], 4, 1, D, 9.0, small=0.02, kind="chain")
    want = c.chain(ctas_per_class=1)
    c.check(*want)
    pg, s = c.table[0, 130 // 16], 130 % 16
    for t in c.dev[2:]:
        t[pg, :, s] = poison
    got = c.chain(ctas_per_class=1)
    for a, b in zip(want, got):
        assert torch.equal(a[:20], b[:20])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("size,sm", [(2.0 ** -120, 1e-9), (2.0 ** -120, 0.1), (2.0 ** 100, 1e-33)])
def test_chains_with_queries_and_scales_at_the_ends_of_the_range(D, size, sm):
    """Scores of next to nothing weigh all keys alike; a masked key's still weigh nothing."""
    c = Sink(57, [40, 3], [9, 30], 4, 2, D, 9.0, small=0.02, kind="chain")
    c.q = (c.q.double() * size).bfloat16()
    c.sm = sm
    c.check(*c.chain())
