"""Offsets of the token history that are not usable for some sequences: the others
are counted all the same, added or rebuilt. The oracle by hand on the host, the
library against it on the GPU."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import step_oracle as S

V = 70
OFFSETS = [
    [0, 2, 5, 3], [0, 2, 1, 4], [0, 3, 6, -1], [-1, 2, 4, 7], [0, 2, 4, 99], [-5, -2, 3, 7],
    [0, 7, 0, 7],                        # two sequences over the same rows, none between
    [5, 3, 7, 2], [2 ** 31 - 1, 0, 7, 7], [3, 3, 3, 3], [0, -2 ** 31, 2 ** 31 - 1, 0],
]


def test_oracle_by_hand():
    z = np.zeros((3, 128))
    s = S.history(z, [9, 9, 9, 9, 9, 9, 9], [0, 2, 5, 3], V)
    assert list(s[:, 9]) == [2, 3, 0]
    assert list(S.history(z, [9] * 7, [0, 3, 6, -1], V)[:, 9]) == [3, 3, 0]
    assert list(S.history(z, [9] * 7, [0, 7, 0, 7], V, accepted=[1, 1, 4])[:, 9]) == [2, 0, 5]


def run(tokens, q, B, state, reset, prompt, accepted):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk

    def i32(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")

    d, st = torch.tensor(state, device="cuda").short(), i32([0])
    sk.splash_token_state_add(i32(tokens), i32(q), d, V, prompt=prompt, reset=reset,
                              accepted=None if accepted is None else i32(accepted), device_status=st)
    bad = any(not 0 <= q[b] <= q[b + 1] <= len(tokens) for b in range(B))
    assert st.item() == (sk.DEVICE_BAD_LENGTH if bad else 0)
    want = S.history(state, tokens, q, V, accepted, prompt, reset)
    assert np.array_equal(d.cpu().numpy(), want)


gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("q", OFFSETS, ids=str)
class TestFewSequences:
    pytestmark = gpu

    def test_added_and_rebuilt(self, q, reset):
        r = np.random.default_rng(3)
        tokens = r.choice([5, 6, -1, V, 69], 7)
        state = r.integers(-32768, 32768, (3, 128))
        state[:, 5] = 32766
        for prompt in (False, True):
            for accepted in (None, [0, 4, -1]):
                run(tokens, q, 3, state, reset, prompt, accepted)


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("B,each", [(40, 50), (600, 3), (2048, 2), (2049, 2), (3000, 1)])
class TestManySequences:
    """Rows of many blocks, offsets in shared memory and not, one, some or no bad
    offset at the ends and inside."""
    pytestmark = gpu

    def test_added_and_rebuilt(self, B, each, reset):
        r = np.random.default_rng(B)
        n = B * each + 2
        tokens = (V * r.random(n) ** 3).astype(np.int64)
        state = np.zeros((B, 128), np.int64)
        good = np.arange(B + 1) * each
        for where, value in ((None, 0), (B, -1), (B, n + 1), (0, -3), (B // 2, 10 ** 9), (B // 2, -7), (1, n - 1)):
            q = good.copy()
            if where is not None:
                q[where] = value
            run(tokens, q.tolist(), B, state, reset, False, None)
        q = good.copy()
        q[r.choice(B + 1, B // 8, replace=False)] = r.integers(-9, n + 9, B // 8)
        # a sequence of thousands of rows over others' would take the oracle long
        wide = np.flatnonzero(np.diff(q) > 500) + 1
        q[wide] = -1
        run(tokens, q.tolist(), B, state, reset, False, r.integers(-1, 4, B))
