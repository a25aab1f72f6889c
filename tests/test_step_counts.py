"""Page counts out of range: no pages, no slots, nothing given back, the count as
it was. On the host the oracle by hand, on the GPU the library against it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import step_oracle as S

COUNTS = [6, -1, 7, 2 ** 31 - 1, -2 ** 31]             # of tables of 5 entries


def scene(count, T1):
    """Sequence 1 of three has the bad count; its row is full of stale entries, 0
    and 2 have pages of their own."""
    table = np.full((3, 5), -1)
    table[0, :1], table[1], table[2, :2] = [10], [10, 11, 12, 13, 14], [11, 12]
    return [3, 4, 20], [2, T1, 5], table, [1, count, 2], [20, 21, 22, 23]


@pytest.mark.parametrize("T1", [1, 30])
@pytest.mark.parametrize("count", COUNTS)
def test_oracle_by_hand(count, T1):
    ctx, T, table, counts, free = scene(count, T1)
    t, c, left, q, new, pos, slots, codes = S.build_tables(ctx, T, table, counts, free, 4, 7 + T1, 30)
    assert np.array_equal(t, table) and c == counts and left == 4 and codes == {S.BAD_LENGTH}
    assert list(slots[:2]) == [163, 164] and set(slots[2:2 + T1]) == {-1}
    assert list(slots[2 + T1:]) == [12 * 16 + i for i in range(4, 9)] and new == [0] * 4
    c, f, n, off, codes = S.release_pages([0, 0, 0], table, counts, free + [-1] * 4, 4)
    assert c == [0, count, 0] and f[:n] == free + [10, 11, 12] and off == [0, 1, 1, 3]
    assert codes == {S.BAD_LENGTH}


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T1", [1, 30, 5000, 0])
@pytest.mark.parametrize("count", COUNTS)
def test_gpu_matches_the_oracle(count, T1, in_place):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk

    def i32(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")

    ctx, T, table, counts, free = scene(count, T1)
    if T1 == 5000:                                       # rows for the second kernel, a table as wide
        table = np.concatenate([table, np.full((3, 320), 9)], 1)
        counts[1] = count = count + 320 if 0 < count < 100 else count
    n = sum(T)
    want = S.build_tables(ctx, T, table, counts, free, 4, n, 30)
    t, c, f, fc = i32(table), i32(counts), i32(free + [-1] * 4), i32([4])
    co, fo = (c, fc) if in_place else (torch.full_like(c, -9), torch.full_like(fc, -9))
    q, new = (torch.full((4,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pos, slots = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    st = i32([0])
    out = {} if in_place else dict(page_counts_out=co, free_count_out=fo)
    sk.splash_build_tables(i32(ctx), i32(T), t, c, f, fc, q, new, pos, slots, 30, device_status=st, **out)
    assert st.item() == S.BAD_LENGTH and co.tolist() == want[1] == counts and fo.item() == want[2] == 4
    assert np.array_equal(t.cpu().numpy(), table) and q.tolist() == want[3] and new.tolist() == want[4]
    assert np.array_equal(pos.cpu().numpy(), want[5]) and np.array_equal(slots.cpu().numpy(), want[6])
    want = S.release_pages([0, 0, 0], table, counts, free + [-1] * 4, 4)
    off = torch.full((4,), -9, dtype=torch.int32, device="cuda")
    st.zero_()
    out = {} if in_place else dict(page_counts_out=co, free_count_out=fo)
    sk.splash_release_pages(i32([0, 0, 0]), t, c, f, fc, off, device_status=st, **out)
    assert st.item() == S.BAD_LENGTH and co.tolist() == want[0] and fo.item() == want[2]
    assert f.tolist() == want[1] and off.tolist() == want[3]
