"""The step operators in the order a verify loop runs them, on the device, eager
and as one captured graph, against the oracles step by step.

The model between is a stand-in of the test: embeddings for q, k and v and an
output head, as torch products. Its logits are what the oracle of the choices
gets, so every integer (tables, slots, choices, accepted lengths, histories) is
compared for equality; the attention goes by the parity bounds."""
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
from oracle import step_oracle as S  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

from gpu_common import assert_parity_scaled  # noqa: E402


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Loop:
    """Static buffers of a batch and one verify step over them."""
    HQ, HKV, D, V, PAGES, MP, MAXT = 8, 2, 128, 1201, 90, 24, 6

    def __init__(self, seed, T):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.B, self.n = len(T), int(sum(T)) + 3                     # three padded rows
        self.T, self.ctx = i32(T), i32(np.zeros(len(T)))
        B, n, V = self.B, self.n, self.V
        self.table = torch.full((B, self.MP), -1, dtype=torch.int32, device="cuda")
        self.counts = i32(np.zeros(B))
        self.free = torch.randperm(self.PAGES, generator=g, device="cuda").int()
        self.fc = i32([self.PAGES])
        self.q_off, self.new = i32(np.zeros(B + 1)), i32(np.zeros(B + 1))
        self.pos, self.slots = i32(np.zeros(n)), i32(np.zeros(n))
        self.pool = sk.alloc_pool(self.PAGES, self.HKV, self.D)
        self.emb = rnd(V, (self.HQ + 2 * self.HKV) * self.D).bfloat16()
        self.head = (rnd(self.HQ * self.D, V) * 0.3).bfloat16()
        self.w = [1 + 0.1 * rnd(self.D) for _ in range(2)]
        self.freq = torch.tensor(1e4 ** (-np.arange(64) / 64), dtype=torch.float32, device="cuda")
        self.x = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.q = torch.zeros(n, self.HQ, self.D, dtype=torch.bfloat16, device="cuda")
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(n, self.HQ, device="cuda")
        self.ws = sk.alloc_workspace(B, n, self.HQ, self.HKV, self.D, self.MAXT)
        self.logits = torch.zeros(n, V, dtype=torch.bfloat16, device="cuda")
        self.tws = sk.alloc_target_workspace(n, V)
        self.targets, self.acc, self.nxt = i32(np.zeros(n)), i32(np.zeros(B)), i32(np.zeros(B))
        self.state = sk.alloc_token_state(B, V)
        self.pen = dict(repetition=torch.full((B,), 1.3, device="cuda"),
                        presence=torch.full((B,), 0.25, device="cuda"),
                        frequency=torch.full((B,), 0.5, device="cuda"))
        self.off = i32(np.zeros(B + 1))
        self.status = i32([0])
        self.scale = self.D ** -0.5

    def step(self):
        sk.splash_build_tables(self.ctx, self.T, self.table, self.counts, self.free, self.fc,
                               self.q_off, self.new, self.pos, self.slots, self.PAGES,
                               device_status=self.status)
        qkv = self.emb[self.x.long()].view(self.n, -1, self.D)
        q, k, v = qkv.split([self.HQ, self.HKV, self.HKV], 1)
        sk.splash_qkv_append(q, k, v, self.q, *self.pool, self.pos, self.slots, inv_freq=self.freq,
                             q_weight=self.w[0], k_weight=self.w[1], device_status=self.status)
        sk.splash_verify_attention(self.q, *self.pool, self.table, self.ctx, self.T, self.scale,
                                   self.MAXT, self.out, self.lse, self.ws, device_status=self.status)
        torch.matmul(self.out.view(self.n, -1), self.head, out=self.logits)
        sk.splash_choose_targets(self.logits, self.q_off, self.targets, self.tws, self.MAXT,
                                 block_tokens=self.x, state=self.state, device_status=self.status,
                                 **self.pen)
        sk.splash_accept_commit(self.x, self.targets, self.T, self.ctx, self.acc, self.nxt,
                                device_status=self.status)
        sk.splash_token_state_add(self.x, self.q_off, self.state, self.V, accepted=self.acc,
                                  device_status=self.status)
        sk.splash_release_pages(self.ctx, self.table, self.counts, self.free, self.fc, self.off,
                                device_status=self.status)

    def tensors(self):
        return [self.ctx, self.table, self.counts, self.free, self.fc, self.q_off, self.pos,
                self.slots, self.q, self.out, self.logits, self.targets, self.acc, self.nxt,
                self.state, *self.pool]


def blocks(loop, step, rng):
    """The next block of every sequence: the token that the last step chose, then
    drafts of which some are the target's."""
    x = rng.integers(0, loop.V, loop.n)
    T, q = loop.T.tolist(), np.concatenate([[0], np.cumsum(loop.T.tolist())])
    if step:
        nxt = loop.nxt.tolist()
        for b in range(loop.B):
            if T[b]:
                x[q[b]] = nxt[b]
    return x


def run_checked(loop, step, rng, pool, K, expect):
    """One step with every result against the oracles."""
    before = dict(ctx=loop.ctx.tolist(), table=loop.table.cpu().numpy(), counts=loop.counts.tolist(),
                  free=loop.free.tolist(), fc=loop.fc.item(), state=loop.state.cpu().numpy())
    T = loop.T.tolist()
    x = loop.x.tolist()
    loop.step()
    torch.cuda.synchronize()
    assert loop.status.item() == 0
    t, counts, left, q, new, pos, slots, codes = S.build_tables(
        before["ctx"], T, before["table"], before["counts"], before["free"], before["fc"], loop.n,
        loop.PAGES)
    assert not codes and loop.q_off.tolist() == q and np.array_equal(loop.table.cpu().numpy(), t)
    assert loop.slots.tolist() == slots.tolist() and loop.pos.tolist() == pos.tolist()
    # the attention, over what the cache holds now
    n = q[-1]
    pool.k_codes[:], pool.v_codes[:] = loop.pool[0].cpu().numpy(), loop.pool[1].cpu().numpy()
    pool.k_scales[:], pool.v_scales[:] = loop.pool[2].cpu().numpy(), loop.pool[3].cpu().numpy()
    o, lse = O.attention(loop.q[:n].double().cpu().numpy(), pool, t, np.array(before["ctx"]),
                         np.array(T), loop.HKV, np.float32(loop.scale))
    assert_parity_scaled(loop.out[:n], loop.lse[:n], o, lse, what=f"step {step}")
    # choices, acceptance, history, from the logits that the GPU has
    z, pick = S.choose(loop.logits.float().cpu().numpy(), q, x, before["state"], [1.3] * loop.B,
                       [0.25] * loop.B, [0.5] * loop.B)
    assert loop.targets[:n].tolist() == pick[:n].tolist()
    acc, ctx, nxt = O.accept_commit(np.array(x[:n]), pick[:n], np.array(T), np.array(before["ctx"]))
    assert loop.acc.tolist() == acc.tolist() and loop.ctx.tolist() == ctx.tolist()
    assert loop.nxt.tolist() == nxt.tolist()
    assert np.array_equal(loop.state.cpu().numpy(),
                          S.history(before["state"], x, q, loop.V, [a if tt else -1 for a, tt in zip(acc, T)]))
    want = S.release_pages(ctx, t, counts, before["free"], left)
    assert loop.counts.tolist() == want[0] and loop.fc.item() == want[2]
    assert loop.free.tolist()[:want[2]] == want[1][:want[2]]
    expect.append([a.clone() for a in loop.tensors()])


T_OF = [4, 1, 0, 6, 3]


def test_a_run_of_steps_matches_the_oracles_and_a_graph_replays_it():
    eager, graphed = Loop(5, T_OF), Loop(5, T_OF)
    pool = O.PagedPool(Loop.PAGES, Loop.HKV, 16, Loop.D)
    rng, expect, inputs = np.random.default_rng(1), [], []
    for step in range(8):
        x = blocks(eager, step, rng)
        if step % 2:                       # drafts that the target will agree with
            eager.x.copy_(i32(x))
            probe = Loop(5, T_OF)
            for a, b in zip(probe.tensors(), eager.tensors()):
                a.copy_(b)
            probe.x.copy_(eager.x)
            probe.step()
            y, q = probe.targets.tolist(), np.concatenate([[0], np.cumsum(T_OF)])
            for b, t in enumerate(T_OF):
                for i in range(1, t):
                    if y[q[b] + i - 1] >= 0:
                        x[q[b] + i] = y[q[b] + i - 1]
                        break              # one accepted draft each
        eager.x.copy_(i32(x))
        inputs.append(x)
        run_checked(eager, step, rng, pool, None, expect)
    assert max(eager.ctx.tolist()) > 8     # drafts were accepted on the way
    # the same steps as replays of one graph
    warm = Loop(5, T_OF)
    warm.step()                            # lets torch's product set itself up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    graphed.x.copy_(i32(inputs[0]))
    with torch.cuda.graph(g):
        graphed.step()
    for step, x in enumerate(inputs):
        graphed.x.copy_(i32(x))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(graphed.tensors(), expect[step]):
            assert torch.equal(a, b), step


def test_running_out_of_pages_in_a_step_leaves_the_served_ones():
    loop = Loop(6, [5, 5, 5])
    loop.fc.fill_(2)                       # pages for two of the three
    loop.x.copy_(i32(np.arange(loop.n)))
    want = Loop(6, [5, 5, 5])
    want.x.copy_(loop.x)
    want.step()
    sk.splash_build_tables(loop.ctx, loop.T, loop.table, loop.counts, loop.free, loop.fc, loop.q_off,
                           loop.new, loop.pos, loop.slots, loop.PAGES, device_status=loop.status)
    assert loop.status.item() == sk.DEVICE_OUT_OF_PAGES
    loop.T.copy_(i32([5, 5, 0]))           # the third sits this step out
    loop.fc.copy_(i32([loop.fc.item()]))
    loop.status.zero_()
    loop.step()
    torch.cuda.synchronize()
    assert loop.status.item() == 0 and loop.acc.tolist()[2] == 0 and loop.nxt.tolist()[2] == -1
    assert loop.ctx.tolist()[2] == 0 and loop.ctx.tolist()[:2] != [0, 0]


def test_two_streams_with_their_own_buffers():
    """The same step on two streams at once: nothing is shared between calls."""
    a, b, ref = Loop(7, T_OF), Loop(7, T_OF), Loop(7, T_OF)
    x = i32(np.random.default_rng(3).integers(0, Loop.V, ref.n))
    for loop in (a, b, ref):
        loop.x.copy_(x)
    ref.step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for loop, s in zip((a, b), streams):
        with torch.cuda.stream(s):
            loop.step()
    torch.cuda.synchronize()
    for loop in (a, b):
        for t, want in zip(loop.tensors(), ref.tensors()):
            assert torch.equal(t, want)
