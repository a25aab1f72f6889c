"""fp64 oracle of the operators that verify a tree of drafts (test infrastructure).

Ancestor masks, attention under a block mask, the accepted path, cached rows moved
together, and log probabilities with entropy and alternatives, each written from its
definition, node by node and row by row. Cached keys come from ``splash_oracle``.
"""
from __future__ import annotations

import numpy as np

from oracle import splash_oracle as O

BAD_LENGTH, BAD_TREE = 2, 6
F32_MAX = float(np.finfo(np.float32).max)


def parent_of(parents, t):
    """(parent, was it usable): a parent that does not come before its node is none."""
    p = int(parents[t])
    return (p, True) if -1 <= p < t else (-1, False)


def ancestors(parents, t):
    """Node t and what it continues, up to the root."""
    up = [t]
    while True:
        p, _ = parent_of(parents, up[-1])
        if p < 0:
            return up
        up.append(p)


def tree_masks(parents, q_offsets, ctx, words):
    """(masks [n, words] uint32, depths, positions, set of device codes)."""
    n = len(parents)
    masks = np.zeros((n, words), np.uint32)
    depths, positions, codes = np.zeros(n, np.int64), np.zeros(n, np.int64), set()
    for b in range(len(q_offsets) - 1):
        lo, hi = int(q_offsets[b]), int(q_offsets[b + 1])
        tree = parents[lo:hi]
        for t in range(hi - lo):
            if not parent_of(tree, t)[1]:
                codes.add(BAD_TREE)
            up = ancestors(tree, t)
            for j in up:
                masks[lo + t, j // 32] |= np.uint32(1 << (j % 32))
            depths[lo + t] = len(up) - 1
            positions[lo + t] = int(ctx[b]) + len(up) - 1
    return masks, depths, positions, codes


def seen_nodes(mask_row, T):
    """Truth value per node of the tree."""
    return np.array([(int(mask_row[j // 32]) >> (j % 32)) & 1 for j in range(T)], bool)


def attention(q, pool, page_table, ctx, T, masks, num_kv_heads, sm_scale):
    """(out, lse, spread) of every row: spread holds what the rounding bounds need,
    sum_j p_j |v_j|, the largest sm_scale * sum_d |q_d k_d| of a seen key, and
    sum_j exp(s_j - max)."""
    q = np.asarray(q, np.float64)
    n, hq, D = q.shape
    G = hq // num_kv_heads
    sm = float(np.float32(sm_scale))
    out, lse = np.zeros((n, hq, D)), np.full((n, hq), -np.inf)
    av, qk, total = np.zeros((n, hq, D)), np.zeros((n, hq)), np.ones((n, hq))
    row = 0
    for b in range(len(T)):
        for h in range(num_kv_heads):
            keys = int(ctx[b]) + int(T[b])
            k, v = O.gather_keys(pool, page_table[b], h, keys)
            for t in range(int(T[b])):
                seen = np.concatenate([np.ones(int(ctx[b]), bool),
                                       seen_nodes(masks[row + t], int(T[b]))])
                if not seen.any():
                    continue
                ks, vs = k[seen], v[seen]
                for g in range(h * G, (h + 1) * G):
                    s = sm * (ks @ q[row + t, g])
                    e = np.exp(s - s.max())
                    total[row + t, g] = e.sum()
                    lse[row + t, g] = s.max() + np.log(e.sum())
                    out[row + t, g] = (e / e.sum()) @ vs
                    av[row + t, g] = (e / e.sum()) @ np.abs(vs)
                    qk[row + t, g] = sm * (np.abs(ks) @ np.abs(q[row + t, g])).max()
        row += int(T[b])
    return out, lse, (av, qk, total)


def accept_tree(tokens, parents, targets, q_offsets, ctx):
    """(accepted, next_tokens, context_lens, path_rows, path_tokens, codes)."""
    n, codes = len(tokens), set()
    acc, nxt, new_ctx = [], [], []
    path_rows, path_tokens = np.full(n, -1, np.int64), np.full(n, -1, np.int64)
    for b in range(len(ctx)):
        lo, hi = int(q_offsets[b]), int(q_offsets[b + 1])
        if hi == lo:
            acc.append(0)
            nxt.append(-1)
            new_ctx.append(int(ctx[b]))
            continue
        for t in range(hi - lo):
            if not parent_of(parents[lo:hi], t)[1]:
                codes.add(BAD_TREE)
        path = [0]
        while True:
            y = int(targets[lo + path[-1]])
            fits = [t for t in range(1, hi - lo) if parent_of(parents[lo:hi], t)[0] == path[-1]
                    and tokens[lo + t] == y and y >= 0]
            if not fits:
                break
            path.append(fits[0])
        for i, t in enumerate(path):
            path_rows[lo + i] = lo + t
            path_tokens[lo + i] = tokens[lo + t]
        acc.append(len(path) - 1)
        nxt.append(int(targets[lo + path[-1]]))
        new_ctx.append(int(ctx[b]) + len(path))
    return acc, nxt, new_ctx, path_rows, path_tokens, codes


def compact(rows, slots, path_rows, q_offsets, accepted):
    """`rows`: what every slot holds (any array with slots first), after the call."""
    old, new = np.array(rows), np.array(rows)
    for b, a in enumerate(accepted):
        o = int(q_offsets[b])
        for i in range(1, int(a) + 1):
            new[slots[o + i]] = old[slots[path_rows[o + i]]]
    return new


def logprobs(z, tokens, k):
    """Row by row: (log p of the token, entropy, k ids, their log p), 64 bits. NaN is
    -inf and infinity the largest fp32."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    n, V = z.shape
    lp, ent = np.full(n, -np.inf), np.zeros(n)
    ids, tops = np.full((n, k), -1, np.int64), np.full((n, k), -np.inf)
    for i in range(n):
        order = sorted(range(V), key=lambda v: (-z[i, v], v))
        x = np.minimum(z[i], F32_MAX)
        if x.max() == -np.inf:
            continue
        e = np.exp(x - x.max())
        p = (x - x.max()) - np.log(e.sum())
        live = e > 0
        ent[i] = -(np.exp(p[live]) * p[live]).sum()
        if 0 <= tokens[i] < V:
            lp[i] = p[tokens[i]]
        for r, v in enumerate(order[:k]):
            if z[i, v] > -np.inf:
                ids[i, r], tops[i, r] = v, p[v]
    return lp, ent, ids, tops
