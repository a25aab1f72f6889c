"""Sequences that get no pages sit a step out, decided on the device: the served
block lengths of the table build against the oracle, and the whole step on a short
free list, with no host read between its calls."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from oracle import splash_oracle as O  # noqa: E402
from oracle import step_oracle as S  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

from test_gpu_step_loop import Loop, i32  # noqa: E402
from test_gpu_step_tables import scene  # noqa: E402


def build_and_check(ctx, T, table, counts, free, have, n, total, in_place):
    served = []
    want = S.build_tables(ctx, T, table, counts, free, have, n, total, served)
    B = len(ctx)
    t, c, f, fc, lens = i32(table), i32(counts), i32(free), i32([have]), i32(T)
    got = lens if in_place else torch.full((B,), -9, dtype=torch.int32, device="cuda")
    q, new = (torch.full((B + 1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pos, slots = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    st = i32([0])
    sk.splash_build_tables(i32(ctx), lens, t, c, f, fc, q, new, pos, slots, total, device_status=st,
                           served_lens=got)
    torch.cuda.synchronize()
    assert got.tolist() == served and (in_place or lens.tolist() == list(T))
    assert np.array_equal(t.cpu().numpy(), want[0]) and c.tolist() == want[1] and fc.item() == want[2]
    assert q.tolist() == want[3] and new.tolist() == want[4]
    assert np.array_equal(pos.cpu().numpy(), want[5]) and np.array_equal(slots.cpu().numpy(), want[6])
    assert st.item() in want[7] if want[7] else st.item() == 0
    return served


# one CTA and two kernels, the scan's chunk edges, offsets kept out of shared memory
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,hi,lens", [(1, 0, [3]), (6, 200, [0, 1, 9, 40]), (128, 300, [0, 5]),
                                       (129, 300, [1, 5]), (1025, 64, [0, 3]), (2500, 40, [0, 1, 4]),
                                       (5, 7000, [1000, 1, 3333]), (300, 500, [16, 40])])
def test_served_lengths_match_the_oracle(B, hi, lens, in_place):
    ctx, T, table, counts, free, total = scene(B + hi, B, hi, lambda r: int(r.choice(lens)))
    n = int(T.sum())
    full = S.build_tables(ctx, T, table, counts, free, len(free), n, total)
    need = len(free) - full[2]
    some = set()
    for have in (0, need // 2, need - 1, need):
        got = build_and_check(ctx, T, table, counts, free[:max(have, 1)], have, n + 5, total, in_place)
        some.add(sum(got) < n)
    assert some == {True, False} or need == 0
    # rows past the caller's count: the last sequences are not served
    build_and_check(ctx, T, table, counts, free, len(free), n - n // 3, total, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_sequences_that_are_not_usable_are_not_served(in_place):
    ctx, T, table, counts, free, total = scene(5, 9, 100, lambda r: 5, max_pages=9)
    ctx[1], T[2], ctx[3], counts[4] = -1, -4, 9 * 16, 77
    table[5, 0] = total                              # out of the pool
    ctx[5], counts[5] = 3, max(counts[5], 1)
    n = int(np.maximum(T, 0).sum())
    got = build_and_check(ctx, T, table, counts, free, len(free), n, total, in_place)
    assert got == [5, 0, 0, 0, 0, 5, 5, 5, 5]
    big = 2 ** 31 - 1
    assert build_and_check([0, 5, 0], [3, big, big], np.full((3, 4), -1), [0, 0, 0], [1, 2], 2, 10, 8,
                           in_place) == [3, 0, 0]
    assert build_and_check([], [], np.zeros((0, 4)), [], [3, 4], 2, 5, 8, in_place) == []


def test_refusals():
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (z(3), z(3), z(3, 5), z(3), z(7), z(1), z(4), z(4), z(9), z(9), 7)
    for bad in (z(4), z(3).float(), z(3).cpu(), z(3, 1), z(6)[::2], 3):
        before = sk.splash_launch_count()
        with pytest.raises((TypeError, ValueError)):
            sk.splash_build_tables(*args, served_lens=bad)
        assert sk.splash_launch_count() == before


class ServedLoop(Loop):
    """Blocks as rows of their own, packed on the device by the step's offsets. All
    sequences are steered to token 7, so that drafts of it are accepted. On the
    host (`by_host`) the served lengths and the tokens are given instead."""

    def __init__(self, seed, T, by_host=False):
        super().__init__(seed, T)
        self.by_host = by_host
        self.asked, self.blocks = self.T.clone(), torch.zeros(self.B, self.MAXT, dtype=torch.int32,
                                                              device="cuda")
        self.bias = dict(bias_offsets=i32(np.arange(self.B + 1)), bias_ids=i32([7] * self.B),
                         bias_values=torch.full((self.B,), 1e4, device="cuda"))

    def step(self):
        tables = (self.table, self.counts, self.free, self.fc, self.q_off, self.new, self.pos,
                  self.slots, self.PAGES)
        if self.by_host:
            sk.splash_build_tables(self.ctx, self.T, *tables, device_status=self.status)
        else:
            sk.splash_build_tables(self.ctx, self.asked, *tables, device_status=self.status,
                                   served_lens=self.T)
            row = torch.arange(self.n, dtype=torch.int32, device="cuda")
            b = (torch.searchsorted(self.q_off, row, right=True) - 1).clamp(max=self.B - 1)
            t = (row - self.q_off[b]).clamp(max=self.MAXT - 1)
            self.x.copy_(torch.where(row < self.q_off[-1], self.blocks[b, t], 0))
        qkv = self.emb[self.x.long()].view(self.n, -1, self.D)
        q, k, v = qkv.split([self.HQ, self.HKV, self.HKV], 1)
        sk.splash_qkv_append(q, k, v, self.q, *self.pool, self.pos, self.slots, inv_freq=self.freq,
                             q_weight=self.w[0], k_weight=self.w[1], device_status=self.status)
        sk.splash_verify_attention(self.q, *self.pool, self.table, self.ctx, self.T, self.scale,
                                   self.MAXT, self.out, self.lse, self.ws, device_status=self.status)
        torch.matmul(self.out.view(self.n, -1), self.head, out=self.logits)
        sk.splash_choose_targets(self.logits, self.q_off, self.targets, self.tws, self.MAXT,
                                 block_tokens=self.x, state=self.state, device_status=self.status,
                                 **self.pen, **self.bias)
        sk.splash_accept_commit(self.x, self.targets, self.T, self.ctx, self.acc, self.nxt,
                                device_status=self.status)
        sk.splash_token_state_add(self.x, self.q_off, self.state, self.V, accepted=self.acc,
                                  device_status=self.status)
        sk.splash_release_pages(self.ctx, self.table, self.counts, self.free, self.fc, self.off,
                                device_status=self.status)


T_OF = [6, 1, 0, 5, 3, 2]


@pytest.mark.parametrize("graph", [False, True])
def test_a_step_on_a_short_free_list_leaves_out_who_gets_no_pages(graph):
    loop, ref = ServedLoop(5, T_OF), ServedLoop(5, T_OF, by_host=True)
    pages = loop.free.tolist()
    reserve = pages[5:]
    for x in (loop, ref):
        x.fc.fill_(5)
    if graph:
        warm = ServedLoop(5, T_OF)
        warm.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loop.step()
        for a, b in zip(loop.tensors(), ref.tensors()):
            assert torch.equal(a, b)                 # a capture runs nothing
    r = np.random.default_rng(2)
    x0, seen = r.integers(8, loop.V, loop.B), set()
    for step in range(18):
        if step == 11:                               # pages come back
            for x in (loop, ref):
                at = x.fc.item()
                x.free[at:at + 40] = i32(reserve[:40])
                x.fc.add_(40)
        blocks = np.where(r.random((loop.B, loop.MAXT)) < 0.6, 7, r.integers(8, loop.V, (loop.B, loop.MAXT)))
        blocks[:, 0] = x0
        before = dict(ctx=loop.ctx.tolist(), state=loop.state.cpu().numpy())
        served = []
        want = S.build_tables(before["ctx"], T_OF, loop.table.cpu().numpy(), loop.counts.tolist(),
                              loop.free.tolist(), loop.fc.item(), loop.n, loop.PAGES, served)
        seen |= {(b, served[b] == T_OF[b]) for b in range(loop.B)}
        # the reference: the others idle by the host, its tokens packed there
        ref.T.copy_(i32(served))
        tokens = np.concatenate([blocks[b, :t] for b, t in enumerate(served)] + [np.zeros(loop.n - sum(served))])
        ref.x.copy_(i32(tokens))
        ref.step()
        loop.blocks.copy_(i32(blocks))
        loop.status.zero_()
        g.replay() if graph else loop.step()
        torch.cuda.synchronize()
        assert loop.status.item() == (sk.DEVICE_OUT_OF_PAGES if served != T_OF else 0)
        assert ref.status.item() == 0 and loop.T.tolist() == served and loop.q_off.tolist() == want[3]
        for a, b in zip(loop.tensors(), ref.tensors()):
            assert torch.equal(a, b), step
        n = sum(served)
        acc, ctx, nxt = O.accept_commit(tokens[:n].astype(int), loop.targets[:n].cpu().numpy(), np.array(served),
                                        np.array(before["ctx"]))
        assert loop.ctx.tolist() == ctx.tolist() and loop.acc.tolist() == acc.tolist()
        assert np.array_equal(loop.state.cpu().numpy(), S.history(
            before["state"], tokens.astype(int), want[3], loop.V, [a if t else -1 for a, t in zip(acc, served)]))
        for b, t in enumerate(served):
            if t:
                x0[b] = nxt[b]
            else:
                assert ctx[b] == before["ctx"][b] and nxt[b] == -1
    # first, middle and last sequences were left out, and all of them served
    assert {(b, True) for b in range(loop.B)} <= seen and len({b for b, ok in seen if not ok}) >= 3
    assert min(c for c, t in zip(loop.ctx.tolist(), T_OF) if t) > 4
