"""Calls of the tree operators that are allowed and rarely made: borders of the plans,
tiny factors, waits that run out, empty batches, several graphs at once."""
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

from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

from test_gpu_tree_attention import Case, i32  # noqa: E402


@pytest.mark.parametrize("B", [511, 512, 513])
@pytest.mark.parametrize("ctas", [0, 1, 9])
def test_the_largest_batch_that_plans_itself_and_the_next(B, ctas):
    rng = np.random.default_rng(B)
    ctx, lens = rng.integers(0, 90, B).tolist(), rng.integers(0, 3, B).tolist()
    ctx[B - 1], lens[0], lens[B - 1] = 700, 0, 2
    c = Case(B, ctx, lens, 4, 1, 64)
    status = i32([0])
    out, lse = c.run(ctas=ctas, status=status, extra=2)
    assert status.item() == 0
    c.check(out, lse)
    assert (out[c.n:] == -3).all() and (lse[c.n:] == -3).all()


@pytest.mark.parametrize("B", [3, 600])
def test_a_batch_without_nodes_writes_nothing(B):
    c = Case(1, [20] * B, [1] * B, 2, 1, 64)
    status = i32([0])
    out, lse = c.run(status=status, block_lens=i32([0] * B))
    assert status.item() == 0 and (out == -3).all() and (lse == -3).all()
    out, lse = c.run(status=status, block_lens=i32([-1] * B))
    assert status.item() == sk.DEVICE_BAD_LENGTH and (out == -3).all() and (lse == -3).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size,sm", [(2.0 ** -120, 1e-9), (2.0 ** -120, 0.1), (2.0 ** 100, 1e-33)])
def test_queries_and_scales_at_the_ends_of_the_range(D, size, sm):
    """Scores of next to nothing weigh all keys alike; a masked key's still weigh nothing."""
    c = Case(21, [40, 3], [9, 70], 4, 2, D)
    c.q = (c.q.double() * size).bfloat16()
    c.sm = sm
    c.check(*c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx,ctas", [(900, 0), (20000, 1), (20000, 0)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(D, ctx, ctas):
    """A wait looks at the clock after two tries, each of which the hardware lets sleep for
    a while: with a limit of 1 ns a call may still pass, and is right then."""
    c = Case(23, [ctx, 64, 5], [40, 3, 17], 8, 2, D)
    for _ in range(3):
        status = i32([0])
        prev = sk.splash_set_wait_limit_ns(1)
        try:
            out, lse = c.run(status=status, ctas=ctas)
            torch.cuda.synchronize()
        finally:
            sk.splash_set_wait_limit_ns(prev)
        print("status", status.item())
        assert status.item() in (0, sk.DEVICE_TIMEOUT)
        if status.item():
            status.zero_()
            out, lse = c.run(status=status, ctas=ctas)
            assert status.item() == 0
        c.check(out, lse)


def test_two_graphs_replayed_side_by_side():
    cases = [Case(31, [700, 9, 300], [30, 60, 5], 8, 2, 128),
             Case(32, [40, 2000], [64, 20], 8, 2, 256)]
    kept = []
    for c in cases:
        a = [i32(c.table), i32(c.ctx), i32(c.lens), i32(c.masks)]
        out = torch.zeros((c.n, c.hq, c.D), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((c.n, c.hq), device="cuda")
        ws = sk.alloc_tree_workspace(len(c.ctx), c.n, c.hq, c.hkv, c.D, c.most)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                sk.splash_verify_attention_tree(c.q, *c.dev, *a, c.sm, c.most, out, lse, ws)
        kept.append((c, g, torch.cuda.Stream(), out, lse, a, ws))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, g, s, *_ in kept:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, _, _, out, lse, *_ in kept:
        c.check(out, lse)
        want = c.run()
        assert torch.equal(want[0], out) and torch.equal(want[1], lse)


@pytest.mark.parametrize("accepted", [2 ** 31 - 1, 6, -2 ** 31])
def test_a_count_past_the_rows_moves_nothing(accepted):
    pool = sk.alloc_pool(3, 2, 64)
    for t in pool:
        t.copy_(torch.randint(-100, 100, t.shape, device="cuda"))
    before = [t.clone() for t in pool]
    status = i32([0])
    sk.splash_kv_compact(*pool, i32([3, 5, 7, 9, 11, 13]), i32([0, 2, 3, 5, -1, -1]), i32([0, 6]),
                         i32([accepted]), device_status=status)
    assert status.item() == (sk.DEVICE_BAD_LENGTH if accepted > 0 else 0)
    for t, b in zip(pool, before):
        assert torch.equal(t, b)


def test_choices_for_a_tree_under_penalties_of_its_committed_tokens():
    """Block tokens of -1 leave the history as it is, whatever the tree's nodes hold."""
    rng = np.random.default_rng(3)
    lens, V = [5, 40, 1], 300
    q = np.concatenate([[0], np.cumsum(lens)])
    n, B = int(q[-1]), len(lens)
    z = rng.standard_normal((n, V)).astype(np.float32)
    state = np.zeros((B, sk.splash_token_state_stride(V)), np.int16)
    state[:, :V] = rng.choice([0, 0, 1, 3, -32768], (B, V))
    rep, pres, freq = (np.array(a, np.float32) for a in ([1.3, 0.8, 1.0], [0.5, 0.0, 0.25],
                                                         [0.25, -0.1, 0.0]))
    f32 = lambda a: torch.tensor(a, device="cuda")  # noqa: E731
    targets, out = i32(np.zeros(n)), torch.zeros((n, V), device="cuda")
    sk.splash_choose_targets(f32(z), i32(q), targets, sk.alloc_target_workspace(n, V), max(lens),
                             block_tokens=i32(np.full(n, -1)), state=f32(state), repetition=f32(rep),
                             presence=f32(pres), frequency=f32(freq), out=out)
    want = np.empty_like(z)
    for b in range(B):
        c = (state[b, :V].astype(np.int32) & 0x7fff).astype(np.float32)
        seen = state[b, :V] != 0
        w = z[q[b]:q[b + 1]]
        w = np.where(seen, np.where(w > 0, w / rep[b], w * rep[b]), w)
        w = w - freq[b] * c
        want[q[b]:q[b + 1]] = np.where(c > 0, w - pres[b], w)
    assert np.array_equal(out.cpu().numpy(), want)
    assert targets.tolist() == want.argmax(1).tolist()
