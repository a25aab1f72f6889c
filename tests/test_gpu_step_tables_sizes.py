"""Table builds and releases on both sides of the sizes at which a second kernel takes
the writes over, for the small and the large scan, against the step oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from oracle import step_oracle as S  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

from test_gpu_step_tables import build, check, i32  # noqa: E402


def split(r, n, B):
    """n rows over B sequences, some without any."""
    cut = np.sort(r.integers(0, n + 1, B - 1))
    return np.diff(np.concatenate([[0], cut, [n]]))


@pytest.mark.parametrize("B", [1, 5, 128, 129, 700])
@pytest.mark.parametrize("n", [1, 1020, 1023, 1024, 1025, 2049, 4095, 4096, 4097, 5003])
def test_build(B, n):
    r = np.random.default_rng(B + n)
    T = split(r, n, B)
    ctx = r.integers(0, 60, B)
    held = [S.pages_of(int(c)) for c in ctx]
    width = max(S.pages_of(int(c + t)) for c, t in zip(ctx, T)) + 1
    total = sum(held) + sum(S.pages_of(int(c + t)) for c, t in zip(ctx, T))
    ids = r.permutation(total)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = ids[at:]
    for have in (len(free), len(free) // 3):
        want = S.build_tables(ctx, T, table, held, free, have, n, total)
        check(build(ctx, T, table, held, free, have, n, total)[0], want)


@pytest.mark.parametrize("B,width", [(1, 1024), (1, 1025), (64, 16), (64, 17), (128, 8), (128, 9),
                                     (129, 8), (256, 16), (256, 17), (700, 5), (700, 6), (16, 1024)])
def test_release(B, width):
    r = np.random.default_rng(B * width)
    counts = r.integers(0, width + 1, B)
    table = np.full((B, width), -1)
    ids, at = r.permutation(int(counts.sum()) + 5), 0
    for b in range(B):
        table[b, :counts[b]] = ids[at:at + counts[b]]
        at += counts[b]
    keep = np.where(r.random(B) < 0.4, 0, r.integers(-1, 16 * width + 20, B))
    for spare in (0, 7, 10 ** 6):
        stack = np.full(min(5 + int(counts.sum()), 5 + spare), -7)
        stack[:5] = ids[at:at + 5]
        want = S.release_pages(keep, table, counts, stack, 5)
        c, fc, f = i32(counts), i32([5]), i32(stack)
        off, st = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda"), i32([0])
        sk.splash_release_pages(i32(keep), i32(table), c, f, fc, off, device_status=st)
        assert c.tolist() == want[0] and f.tolist() == want[1] and fc.item() == want[2]
        assert off.tolist() == want[3] and st.item() == (S.BAD_LENGTH if want[4] else 0)
