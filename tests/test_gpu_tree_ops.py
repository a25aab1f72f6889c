"""Masks, accepted paths and moved cache rows of trees of drafts on the GPU against
the oracle: whole numbers and bit patterns, so everything by equality."""
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

from oracle import tree_oracle as T  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402


def i32(a):
    return torch.tensor(np.asarray(a), device="cuda").to(torch.int32)


def trees(rng, lens, back):
    return np.array([t - 1 - int(rng.integers(0, min(back, t))) if t else -1
                     for n in lens for t in range(n)], np.int64)


LENS = [[1], [2, 0, 3], [32], [33, 1], [64, 31, 65], [128, 0, 0, 127], [256, 255, 129, 1],
        [7] * 300]


@pytest.mark.parametrize("lens", LENS, ids=[str(x[:4]) for x in LENS])
@pytest.mark.parametrize("back", [1, 4, 300])
def test_masks(lens, back):
    rng = np.random.default_rng(len(lens) * 7 + back)
    off = np.concatenate([[0], np.cumsum(lens)])
    parents = trees(rng, lens, back)
    ctx = rng.integers(0, 1000, len(lens))
    if len(parents) > 2:                               # a second root
        parents[off[len(lens)] - 1] = -1
    words, most = -(-max(lens) // 32) + 1, max(lens)
    n = len(parents)
    masks = torch.full((n + 2, words), 77, dtype=torch.int32, device="cuda")
    depths, pos = i32(np.full(n + 2, -9)), i32(np.full(n + 2, -9))
    status = i32([0])
    more = i32(np.concatenate([parents, [5, 5]]))      # rows behind the last sequence
    sk.splash_tree_masks(more, i32(off), masks, most, context_lens=i32(ctx), depths=depths,
                         positions=pos, device_status=status)
    want, d, p, codes = T.tree_masks(parents, off, ctx, words - 1)
    assert status.item() == 0 and not codes
    assert np.array_equal(masks[:n, :-1].cpu().numpy().view(np.uint32), want)
    assert depths.tolist() == d.tolist() + [-9, -9] and pos.tolist() == p.tolist() + [-9, -9]
    assert (masks[n:] == 77).all() and (masks[:, -1] == 77).all()
    only = torch.full_like(masks, 77)
    sk.splash_tree_masks(more, i32(off), only, most)   # the masks alone
    assert torch.equal(only, masks)


def test_masks_of_bad_parents_and_offsets():
    parents = i32([-1, 1, 0, 3, -7, 4, 2 ** 31 - 1])
    masks, status = torch.zeros((7, 1), dtype=torch.int32, device="cuda"), i32([0])
    sk.splash_tree_masks(parents, i32([0, 7]), masks, 7, device_status=status)
    want, _, _, codes = T.tree_masks(parents.tolist(), [0, 7], [0], 1)
    assert status.item() == sk.DEVICE_BAD_TREE and codes == {T.BAD_TREE}
    assert masks[:, 0].tolist() == want[:, 0].tolist()
    # sequences with unusable offsets are left, the others are done
    for off in ([0, 3, 2, 7], [0, 3, 9, 7], [-2, 3, 3, 7]):
        masks.fill_(5)
        status.zero_()
        sk.splash_tree_masks(i32([-1, 0, 1] * 3)[:7].contiguous(), i32(off), masks, 5,
                             device_status=status)
        assert status.item() == sk.DEVICE_BAD_LENGTH
    status.zero_()
    masks.fill_(5)
    sk.splash_tree_masks(i32([-1, 0, 0, -1, 0, 1, 2]), i32([0, 3, 7]), masks, 3,
                         device_status=status)
    assert status.item() == sk.DEVICE_BAD_LENGTH
    assert masks[:, 0].tolist() == [1, 3, 5, 5, 5, 5, 5]


def accept_case(rng, lens, back, vocab):
    parents = trees(rng, lens, back)
    n = len(parents)
    tokens, targets = rng.integers(0, vocab, n), rng.integers(0, vocab, n)
    off = np.concatenate([[0], np.cumsum(lens)])
    for b, m in enumerate(lens):                       # half of the trees are agreed with
        for t in range(1, m):
            if b % 2 == 0 and rng.random() < 0.8:
                targets[off[b] + parents[off[b] + t]] = tokens[off[b] + t]
    return parents, tokens, targets, off


@pytest.mark.parametrize("lens", LENS, ids=[str(x[:4]) for x in LENS])
@pytest.mark.parametrize("back,vocab", [(1, 2), (3, 4), (300, 3), (2, 50000)])
def test_accept(lens, back, vocab):
    rng = np.random.default_rng(len(lens) * 31 + back + vocab)
    parents, tokens, targets, off = accept_case(rng, lens, back, vocab)
    if len(tokens) > 8:
        tokens[5], targets[7] = -1, -1                 # a node and a choice that are none
    ctx = rng.integers(0, 1000, len(lens))
    n, B = len(parents), len(lens)
    out = {k: i32(np.full(m, -9)) for k, m in dict(acc=B, nxt=B, rows=n + 2, toks=n + 2).items()}
    pad = lambda a: i32(np.concatenate([a, [1, 1]]))  # noqa: E731
    c, status = i32(ctx), i32([0])
    sk.splash_accept_tree(pad(tokens), pad(parents), pad(targets), i32(off), c, out["acc"],
                          out["nxt"], out["rows"], out["toks"], max(lens), device_status=status)
    acc, nxt, new, rows, toks, _ = T.accept_tree(tokens, parents, targets, off, ctx)
    assert status.item() == 0
    assert out["acc"].tolist() == acc and out["nxt"].tolist() == nxt and c.tolist() == new
    assert out["rows"].tolist() == rows.tolist() + [-9, -9]
    assert out["toks"].tolist() == toks.tolist() + [-9, -9]
    other, before = i32(np.zeros(B)), i32(ctx)         # lengths into another tensor, no tokens
    sk.splash_accept_tree(pad(tokens), pad(parents), pad(targets), i32(off), before, out["acc"],
                          out["nxt"], out["rows"], None, max(lens), context_lens_out=other)
    assert other.tolist() == new and before.tolist() == ctx.tolist()


def test_accept_with_bad_parents_and_offsets():
    status, acc, nxt = i32([0]), i32([7, 7]), i32([7, 7])
    rows, toks = i32(np.full(6, 7)), i32(np.full(6, 7))
    ctx = i32([10, 20])
    tokens, targets = i32([1, 2, 2, 1, 2, 3]), i32([2, 2, 2, 2, 3, 9])
    sk.splash_accept_tree(tokens, i32([-1, 1, 0, -1, 0, 1]), targets, i32([0, 3, 6]), ctx, acc, nxt,
                          rows, toks, 3, device_status=status)
    assert status.item() == sk.DEVICE_BAD_TREE
    assert acc.tolist() == [1, 2] and nxt.tolist() == [2, 9] and ctx.tolist() == [12, 23]
    assert rows.tolist() == [0, 2, -1, 3, 4, 5] and toks.tolist() == [1, 2, -1, 1, 2, 3]
    status.zero_()
    rows.fill_(7)
    sk.splash_accept_tree(tokens, i32([-1, 0, 0, -1, 0, 1]), targets, i32([0, 8, 6]), ctx, acc, nxt,
                          rows, toks, 3, device_status=status)
    assert status.item() == sk.DEVICE_BAD_LENGTH and acc.tolist() == [0, 0]
    assert nxt.tolist() == [-1, -1] and ctx.tolist() == [12, 23] and (rows == 7).all()


def compact_case(rng, lens, layers, hkv, D, share=0.4):
    off = np.concatenate([[0], np.cumsum(lens)])
    n = int(off[-1])
    pages = n // 16 + 4
    slots = rng.permutation(pages * 16)[:n]
    path, acc = np.full(n, -1, np.int64), []
    for b, m in enumerate(lens):
        nodes = [t for t in range(m) if t == 0 or rng.random() < share]
        path[off[b]:off[b] + len(nodes)] = off[b] + np.array(nodes, np.int64)
        acc.append(max(0, len(nodes) - 1))
    pool = sk.alloc_pool(pages, hkv, D, num_layers=layers)
    g = torch.Generator(device="cuda").manual_seed(n)
    for t in pool[:2]:
        t.copy_(torch.randint(-128, 128, t.shape, generator=g, device="cuda"))
    for t in pool[2:]:
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    return off, slots, path, acc, pool


def by_slot(t):
    """The pool tensor with slots first: (page, place in page) -> row of all the rest."""
    a = t.cpu().numpy() if t.dtype is torch.int8 else t.cpu().numpy().view(np.int32)
    if t.dtype is torch.int8:                          # [L, pages, H, P, D]
        a = a.transpose(1, 3, 0, 2, 4)
    else:
        a = a.transpose(1, 3, 0, 2)
    return a.reshape(-1, *a.shape[2:])


@pytest.mark.parametrize("lens", LENS, ids=[str(x[:4]) for x in LENS])
@pytest.mark.parametrize("layers,hkv,D", [(1, 1, 64), (3, 2, 128), (2, 3, 256), (5, 1, 128)])
@pytest.mark.parametrize("share", [0.15, 0.8])
def test_compact(lens, layers, hkv, D, share):
    rng = np.random.default_rng(len(lens) + layers * 10)
    off, slots, path, acc, pool = compact_case(rng, lens, layers, hkv, D, share)
    want = [T.compact(by_slot(t), slots, path, off, acc) for t in pool]
    status = i32([0])
    sk.splash_kv_compact(*pool, i32(slots), i32(path), i32(off), i32(acc), device_status=status)
    assert status.item() == 0
    for t, w in zip(pool, want):
        assert np.array_equal(by_slot(t), w)


def test_compact_of_one_pool_and_of_layers_with_gaps():
    rng = np.random.default_rng(3)
    off, slots, path, acc, pool = compact_case(rng, [20, 9], 4, 2, 128)
    want = [T.compact(by_slot(t), slots, path, off, acc) for t in pool]
    single = [t[1] for t in pool]                      # a layer's own views
    before = [t.clone() for t in pool]
    sk.splash_kv_compact(*single, i32(slots), i32(path), i32(off), i32(acc))
    for t, w, b in zip(pool, want, before):
        got = by_slot(t)
        assert np.array_equal(got[:, 1], w[:, 1])
        assert torch.equal(t[0], b[0]) and torch.equal(t[2:], b[2:])
    for t, b in zip(pool, before):
        t.copy_(b)
    sk.splash_kv_compact(pool[0][::2], pool[1][::2], pool[2][::2].contiguous(),
                         pool[3][::2].contiguous(), i32(slots), i32(path), i32(off), i32(acc))
    for t, w, b in zip(pool[:2], want[:2], before[:2]):
        got = by_slot(t)
        assert np.array_equal(got[:, ::2], w[:, ::2]) and torch.equal(t[1::2], b[1::2])


def test_compact_refuses_rows_by_rows():
    rng = np.random.default_rng(4)
    off, slots, path, acc, pool = compact_case(rng, [12, 12], 1, 1, 64, share=0.0)
    path[:4], path[12:15] = [0, 3, 5, 9], [12, 14, 17]
    acc = [3, 2]
    before = [by_slot(t) for t in pool]

    def run(code, expect_path=None, p=path, s=slots, a=acc, o=off):
        for t, b in zip(pool, before):
            shape = (t.shape[1], 16, t.shape[0], t.shape[2]) + tuple(t.shape[4:])
            back = torch.tensor(b.reshape(shape), device="cuda")
            if t.dtype is not torch.int8:
                back = back.view(torch.float32)
            t.copy_(back.permute(2, 0, 3, 1, *range(4, back.dim())))
        status = i32([0])
        sk.splash_kv_compact(*pool, i32(s), i32(p), i32(o), i32(a), device_status=status)
        assert status.item() == code
        return [by_slot(t) for t in pool]

    def moved(pairs):
        out = []
        for b in before:
            w = b.copy()
            for dst, src in pairs:
                w[slots[dst]] = b[slots[src]]
            out.append(w)
        return out

    def same(x, y):
        return all(np.array_equal(p, q) for p, q in zip(x, y))

    assert same(run(0), moved([(1, 3), (2, 5), (3, 9), (13, 14), (14, 17)]))
    # a path row before its place, of another sequence, none
    for bad in (1, 12, -1, 10 ** 6):
        p = path.copy()
        p[2] = bad
        assert same(run(sk.DEVICE_BAD_TREE, p=p), moved([(1, 3), (3, 9), (13, 14), (14, 17)]))
    # slots past the pool and none
    for at in (2, 5):
        s = slots.copy()
        s[at] = pool[0].shape[1] * 16
        assert same(run(sk.DEVICE_BAD_PAGE, s=s), moved([(1, 3), (3, 9), (13, 14), (14, 17)]))
        s[at] = -1
        assert same(run(0, s=s), moved([(1, 3), (3, 9), (13, 14), (14, 17)]))
    # counts past the rows; none accepted
    assert same(run(sk.DEVICE_BAD_LENGTH, a=[12, 2]), moved([(13, 14), (14, 17)]))
    assert same(run(sk.DEVICE_BAD_LENGTH, a=[2 ** 31 - 2, 2]), moved([(13, 14), (14, 17)]))
    assert same(run(0, a=[0, -3]), moved([]))
    assert same(run(sk.DEVICE_BAD_LENGTH, o=[0, 12, 30]), moved([(1, 3), (2, 5), (3, 9)]))


def test_compact_past_four_gigabytes():
    D, hkv = 256, 4
    pages = 2 ** 32 // (hkv * 2 * 16 * D) + 4
    codes = torch.zeros((2, pages, hkv, 2, 16, D), dtype=torch.int8, device="cuda")
    ks, vs = (torch.zeros((2, pages, hkv, 16), device="cuda") for _ in range(2))
    last = pages * 16 - 1
    codes[:, -1, :, :, 15], ks[:, -1, :, 15], vs[:, -1, :, 15] = 7, 2.0, 3.0
    sk.splash_kv_compact(codes[..., 0, :, :], codes[..., 1, :, :], ks, vs,
                         i32([last - 40, last - 17, last]), i32([0, 2, -1]), i32([0, 3]), i32([1]))
    page, at = (last - 17) // 16, (last - 17) % 16
    assert (codes[:, page, :, :, at] == 7).all() and (ks[:, page, :, at] == 2).all()
    assert (vs[:, page, :, at] == 3).all() and int(codes[:, :64].int().abs().sum()) == 0
    assert int((codes.view(2, pages, -1) != 0).any(-1).sum()) == 4
