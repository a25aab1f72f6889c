"""A verify loop over trees of drafts, all on the device: tables, masks, append,
attention, choices, accepted path, moved cache rows, history, release and log
probabilities, eager and as one captured graph.

The model between is a stand-in of the test (embeddings and an output head as torch
products). Every whole number is compared with the oracles, the cache with what a
chain of the committed tokens puts into it, bit for bit."""
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
from oracle import tree_oracle as T  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

from gpu_common import assert_parity_scaled  # noqa: E402


def i32(a):
    return torch.tensor(np.asarray(a), device="cuda").to(torch.int32)


class Loop:
    """Static buffers of a batch, two layers, one step over them."""
    HQ, HKV, D, V, PAGES, MP, MAXT, L, K = 8, 2, 128, 601, 90, 24, 40, 2, 4

    def __init__(self, seed, lens):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        B, n, V = len(lens), int(sum(lens)) + 3, self.V              # three padded rows
        zeros = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.B, self.n = B, n
        self.lens, self.ctx = i32(lens), zeros(B)
        self.table = torch.full((B, self.MP), -1, dtype=torch.int32, device="cuda")
        self.counts, self.fc = zeros(B), i32([self.PAGES])
        self.free = torch.randperm(self.PAGES, generator=g, device="cuda").int()
        self.q_off, self.new, self.off = zeros(B + 1), zeros(B + 1), zeros(B + 1)
        self.order, self.slots, self.pos, self.depth = zeros(n), zeros(n), zeros(n), zeros(n)
        self.pool = sk.alloc_pool(self.PAGES, self.HKV, self.D, num_layers=self.L)
        self.emb = rnd(V, self.L, (self.HQ + 2 * self.HKV) * self.D).bfloat16()
        self.head = (rnd(self.HQ * self.D, V) * 0.3).bfloat16()
        self.freq = torch.tensor(1e4 ** (-np.arange(64) / 64), dtype=torch.float32, device="cuda")
        self.x, self.parents, self.masks = zeros(n), zeros(n), zeros(n, 2)
        self.q = [zeros(n, self.HQ, self.D, dtype=torch.bfloat16) for _ in range(self.L)]
        self.out = [torch.zeros_like(self.q[0]) for _ in range(self.L)]
        self.lse = zeros(n, self.HQ, dtype=torch.float32)
        self.ws = sk.alloc_tree_workspace(B, n, self.HQ, self.HKV, self.D, self.MAXT)
        self.logits = zeros(n, V, dtype=torch.bfloat16)
        self.tws = sk.alloc_target_workspace(n, V)
        self.targets, self.acc, self.nxt = zeros(n), zeros(B), zeros(B)
        self.path, self.path_tok = zeros(n) - 1, zeros(n) - 1
        self.state = sk.alloc_token_state(B, V)
        self.lws = sk.alloc_logprobs_workspace(n, V)
        self.lp, self.ent = zeros(n, dtype=torch.float32), zeros(n, dtype=torch.float32)
        self.ids, self.tops = zeros(n, self.K), zeros(n, self.K, dtype=torch.float32)
        self.status = zeros(1)
        self.scale = self.D ** -0.5

    def step(self):
        st = dict(device_status=self.status)
        sk.splash_build_tables(self.ctx, self.lens, self.table, self.counts, self.free, self.fc,
                               self.q_off, self.new, self.order, self.slots, self.PAGES, **st)
        sk.splash_tree_masks(self.parents, self.q_off, self.masks, self.MAXT,
                             context_lens=self.ctx, depths=self.depth, positions=self.pos, **st)
        qkv = self.emb[self.x.long()].view(self.n, self.L, -1, self.D)
        for l in range(self.L):
            layer = [t[l] for t in self.pool]
            q, k, v = qkv[:, l].split([self.HQ, self.HKV, self.HKV], 1)
            sk.splash_qkv_append(q, k, v, self.q[l], *layer, self.pos, self.slots,
                                 inv_freq=self.freq, **st)
            sk.splash_verify_attention_tree(self.q[l], *layer, self.table, self.ctx, self.lens,
                                            self.masks, self.scale, self.MAXT, self.out[l],
                                            self.lse, self.ws, **st)
        torch.matmul((self.out[0] + self.out[1]).view(self.n, -1), self.head, out=self.logits)
        sk.splash_choose_targets(self.logits, self.q_off, self.targets, self.tws, self.MAXT, **st)
        sk.splash_accept_tree(self.x, self.parents, self.targets, self.q_off, self.ctx, self.acc,
                              self.nxt, self.path, self.path_tok, self.MAXT, **st)
        sk.splash_kv_compact(*self.pool, self.slots, self.path, self.q_off, self.acc, **st)
        sk.splash_token_state_add(self.path_tok, self.q_off, self.state, self.V, accepted=self.acc,
                                  **st)
        sk.splash_release_pages(self.ctx, self.table, self.counts, self.free, self.fc, self.off, **st)
        sk.splash_token_logprobs(self.logits, self.lws, tokens=self.targets, logprobs=self.lp,
                                 entropy=self.ent, top_ids=self.ids, top_logprobs=self.tops,
                                 rows=self.path, **st)

    def tensors(self):
        return [self.ctx, self.table, self.counts, self.free, self.fc, self.q_off, self.slots,
                self.pos, self.depth, self.masks, *self.q, *self.out, self.lse, self.logits,
                self.targets, self.acc, self.nxt, self.path, self.path_tok, self.state, self.lp,
                self.ent, self.ids, self.tops, *self.pool]


def check_step(loop, step, committed):
    before = dict(ctx=loop.ctx.tolist(), table=loop.table.cpu().numpy(), counts=loop.counts.tolist(),
                  free=loop.free.tolist(), fc=loop.fc.item(), state=loop.state.cpu().numpy())
    lens, x, parents = loop.lens.tolist(), loop.x.tolist(), loop.parents.tolist()
    # what the cache holds when the attention runs: a step without the moves
    probe = Loop(5, lens)
    for a, b in zip(probe.tensors(), loop.tensors()):
        a.copy_(b)
    probe.x.copy_(loop.x)
    probe.parents.copy_(loop.parents)
    loop.step()
    torch.cuda.synchronize()
    assert loop.status.item() == 0
    t, counts, left, q, new, _, slots, codes = S.build_tables(
        before["ctx"], lens, before["table"], before["counts"], before["free"], before["fc"], loop.n,
        loop.PAGES)
    assert not codes and np.array_equal(loop.table.cpu().numpy(), t)
    assert loop.slots.tolist() == slots.tolist()
    n = q[-1]
    m, d, pos, codes = T.tree_masks(parents[:n], q, before["ctx"], 2)
    assert not codes and np.array_equal(loop.masks[:n].cpu().numpy().view(np.uint32), m)
    assert loop.pos.tolist()[:n] == pos.tolist()
    acc, nxt, ctx, rows, toks, codes = T.accept_tree(x[:n], parents[:n], loop.targets.tolist(), q,
                                                     before["ctx"])
    assert not codes and loop.acc.tolist() == acc and loop.nxt.tolist() == nxt
    assert loop.ctx.tolist() == ctx and loop.path.tolist()[:n] == rows.tolist()
    assert loop.path_tok.tolist()[:n] == toks.tolist()
    assert np.array_equal(loop.state.cpu().numpy(),
                          S.history(before["state"], toks.tolist() + [0] * 3, q, loop.V,
                                    [a if k else -1 for a, k in zip(acc, lens)]))
    want = S.release_pages(ctx, t, counts, before["free"], left)
    assert loop.counts.tolist() == want[0] and loop.fc.item() == want[2]
    # the committed tokens lie in the cache in order, as a chain's append puts them there
    for b in range(loop.B):
        committed[b] += [int(toks[q[b] + i]) for i in range(acc[b] + 1)] if lens[b] else []
        assert len(committed[b]) == ctx[b]
    chain = sk.alloc_pool(loop.PAGES, loop.HKV, loop.D, num_layers=loop.L)
    for b in range(loop.B):
        if not ctx[b]:
            continue
        tok = i32(committed[b]).long()
        j = np.arange(ctx[b])
        at = i32(t[b][j // 16] * 16 + j % 16)
        rowsx = loop.emb[tok].view(ctx[b], loop.L, -1, loop.D)
        for l in range(loop.L):
            qq, k, v = rowsx[:, l].split([loop.HQ, loop.HKV, loop.HKV], 1)
            sk.splash_qkv_append(qq, k, v, torch.empty_like(qq).contiguous(),
                                 *[p[l] for p in chain], i32(j), at, inv_freq=loop.freq)
        pg, sl = (at // 16).long(), (at % 16).long()
        for got, ref in zip(loop.pool, chain):
            assert torch.equal(got[:, pg, :, sl], ref[:, pg, :, sl]), (step, b)
    # log probabilities of what was emitted
    lp, ent, ids, tops = T.logprobs(loop.logits.double().cpu().numpy(), loop.targets.tolist(), loop.K)
    for i, r in enumerate(rows):
        if r >= 0:
            assert abs(loop.lp[i].item() - lp[r]) < 1e-5 and abs(loop.ent[i].item() - ent[r]) < 1e-4
            assert loop.ids[i].tolist() == ids[r].tolist()
    # the attention of the first layer, over the cache before the rows were moved
    l0 = [p[0] for p in probe.pool]
    qkv = probe.emb[probe.x.long()].view(probe.n, probe.L, -1, probe.D)[:, 0]
    qq, k, v = qkv.split([loop.HQ, loop.HKV, loop.HKV], 1)
    sk.splash_qkv_append(qq, k, v, probe.q[0], *l0, loop.pos, loop.slots, inv_freq=loop.freq)
    pool = O.PagedPool(loop.PAGES, loop.HKV, 16, loop.D)
    pool.k_codes, pool.v_codes = l0[0].cpu().numpy(), l0[1].cpu().numpy()
    pool.k_scales, pool.v_scales = l0[2].cpu().numpy(), l0[3].cpu().numpy()
    o, lse, _ = T.attention(loop.q[0][:n].double().cpu().numpy(), pool, t, before["ctx"], lens, m,
                            loop.HKV, loop.scale)
    assert_parity_scaled(loop.out[0][:n], torch.tensor(lse), o, lse, what=f"step {step}")


LENS = [12, 1, 0, 33, 5]


def trees(loop, rng, known):
    """Random trees; where the target's choices are known, some of them among the nodes."""
    q = np.concatenate([[0], np.cumsum(LENS)])
    x, parents = rng.integers(0, loop.V, loop.n), np.full(loop.n, -1)
    for b, m in enumerate(LENS):
        for t in range(1, m):
            parents[q[b] + t] = max(0, t - 1 - int(rng.integers(0, 3)))
        if m:
            x[q[b]] = known[b]
    return x, parents


def test_a_run_of_steps_matches_the_oracles_and_a_graph_replays_it():
    eager, rng = Loop(5, LENS), np.random.default_rng(1)
    committed, inputs, expect = [[] for _ in LENS], [], []
    q = np.concatenate([[0], np.cumsum(LENS)])
    deepest = 0
    for step in range(5):
        known = [max(0, v) for v in eager.nxt.tolist()] if step else [7] * len(LENS)
        x, parents = trees(eager, rng, known)
        for _ in range(4):                 # nodes that the target will agree with, a level at a time
            probe = Loop(5, LENS)
            for a, b in zip(probe.tensors(), eager.tensors()):
                a.copy_(b)
            probe.x.copy_(i32(x))
            probe.parents.copy_(i32(parents))
            probe.step()
            y = probe.targets.tolist()
            for b, m in enumerate(LENS):
                last = probe.path.tolist()[q[b]:q[b] + m]
                last = [r for r in last if r >= 0]
                kids = [t for t in range(1, m) if last and parents[q[b] + t] == last[-1] - q[b]]
                if kids:
                    x[q[b] + kids[-1]] = y[last[-1]]
        eager.x.copy_(i32(x))
        eager.parents.copy_(i32(parents))
        inputs.append((x, parents))
        check_step(eager, step, committed)
        deepest = max(deepest, *eager.acc.tolist())
        expect.append([t.clone() for t in eager.tensors()])
    assert deepest >= 2 and max(eager.ctx.tolist()) > 12
    graphed = Loop(5, LENS)
    warm = Loop(5, LENS)
    warm.step()
    torch.cuda.synchronize()
    graphed.x.copy_(i32(inputs[0][0]))
    graphed.parents.copy_(i32(inputs[0][1]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.step()
    for step, (x, parents) in enumerate(inputs):
        graphed.x.copy_(i32(x))
        graphed.parents.copy_(i32(parents))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(graphed.tensors(), expect[step]):
            assert torch.equal(a, b), step


def test_two_streams_with_their_own_buffers():
    loops = [Loop(7, LENS) for _ in range(3)]
    x, parents = trees(loops[0], np.random.default_rng(3), [1] * len(LENS))
    for loop in loops:
        loop.x.copy_(i32(x))
        loop.parents.copy_(i32(parents))
    loops[2].step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for loop, s in zip(loops, streams):
        with torch.cuda.stream(s):
            loop.step()
    torch.cuda.synchronize()
    for loop in loops[:2]:
        for t, want in zip(loop.tensors(), loops[2].tensors()):
            assert torch.equal(t, want)
