"""What the tree operators report: unusable offsets whatever else the call holds, and waits
that run out."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

from test_gpu_tree_attention import Case, i32  # noqa: E402


@pytest.mark.parametrize("offsets", [[0, 9, 4], [0, 3, 2], [-1, 2, 6], [0, 2, 7]])
@pytest.mark.parametrize("accepted", [[0, 0], [0, 1], [-5, 0], [2, 0]])
def test_unusable_offsets_are_reported_whatever_was_accepted(offsets, accepted):
    pool = sk.alloc_pool(3, 2, 64)
    for t in pool:
        t.copy_(torch.randint(-100, 100, t.shape, device="cuda"))
    before = [t.clone() for t in pool]
    status = i32([0])
    # the second sequence's path moves nothing: its nodes lie where they belong
    sk.splash_kv_compact(*pool, i32([3, 5, 7, 9, 11, 13]), i32([0, 1, 2, 3, 4, 5]), i32(offsets),
                         i32(accepted), device_status=status)
    assert status.item() == sk.DEVICE_BAD_LENGTH
    for t, b in zip(pool, before):
        assert torch.equal(t, b)


def test_what_accept_writes_for_unusable_offsets_is_reported_by_compact_too():
    tokens, parents = i32([1, 2, 3]), i32([-1, 0, 1])
    offsets, ctx = i32([0, 4]), i32([7])
    acc, nxt, rows, status = i32([9]), i32([9]), i32([9, 9, 9]), i32([0])
    sk.splash_accept_tree(tokens, parents, i32([2, 3, 4]), offsets, ctx, acc, nxt, rows, None, 3,
                          device_status=status)
    assert (status.item(), acc.item(), nxt.item(), ctx.item()) == (sk.DEVICE_BAD_LENGTH, 0, -1, 7)
    assert rows.tolist() == [9, 9, 9]
    status.zero_()
    sk.splash_kv_compact(*sk.alloc_pool(2, 1, 64), i32([1, 2, 3]), rows, offsets, acc,
                         device_status=status)
    assert status.item() == sk.DEVICE_BAD_LENGTH


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_runs_out_within_a_few_calls(D):
    """One CTA, 20000 keys and a limit of 1 ns: hundreds of waits for copies and for other
    roles. The hardware may let each sleep past the clock's first look, all of them in six
    calls no. Each such call reports it, and the next with the usual limit is as before."""
    c = Case(23, [20000, 64, 5], [40, 3, 17], 8, 2, D)
    want, status, ran_out = c.run(ctas=1), i32([0]), 0
    for _ in range(6):
        status.zero_()
        prev = sk.splash_set_wait_limit_ns(1)
        try:
            c.run(status=status, ctas=1)
            torch.cuda.synchronize()
        finally:
            sk.splash_set_wait_limit_ns(prev)
        assert status.item() in (0, sk.DEVICE_TIMEOUT)
        ran_out += status.item() == sk.DEVICE_TIMEOUT
        status.zero_()
        got = c.run(status=status, ctas=1)
        assert status.item() == 0
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert ran_out
