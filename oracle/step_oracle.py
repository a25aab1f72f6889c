"""fp64 oracle of the operators around verify attention (test infrastructure).

Page tables and slot maps, release of pages, the q/k norm and rotation, cached
rows by slot, the target's choices and the token history, each written from its
definition, sequence by sequence and value by value where that is the plainest
way. The quantiser is ``splash_oracle``'s.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

PAGE = 16
BAD_PAGE, BAD_LENGTH, OUT_OF_PAGES = 1, 2, 5


def pages_of(tokens: int) -> int:
    return -(-tokens // PAGE)


def build_tables(ctx, T, table, counts, free, free_count, num_tokens, num_pages, served=None):
    """(table, counts, free_count, q_offsets, new_offsets, positions, slots,
    set of device codes) after the call; the inputs are not changed. With a list
    `served`, that list gets the served block lengths, and the rows are packed by
    them."""
    table, counts = np.array(table, np.int64), [int(c) for c in counts]
    B, max_pages = len(ctx), table.shape[1]
    codes = set()
    stack = [int(p) for p in free[:max(0, min(int(free_count), len(free)))]]
    q_off, new_off = [0], [0]
    pos, slots = np.zeros(num_tokens, np.int64), np.full(num_tokens, -1, np.int64)
    asked = asked_rows = 0          # pages and rows that this and earlier sequences want
    had = len(stack)
    for b in range(B):
        c, t, have = int(ctx[b]), int(T[b]), counts[b]
        rows = max(t, 0)
        bad = t < 0 or c < 0 or c + t > max_pages * PAGE or not 0 <= have <= max_pages
        if bad:
            codes.add(BAD_LENGTH)
        need = 0 if bad or rows == 0 else max(0, pages_of(c + t) - have)
        asked += need
        asked_rows += rows
        fits = asked_rows <= num_tokens
        if rows and not fits:
            codes.add(BAD_LENGTH)
        got = 0
        if need and fits and asked <= had:
            for j in range(have, have + need):
                page = stack.pop()
                if not 0 <= page < num_pages:
                    codes.add(BAD_PAGE)
                table[b, j] = page
            got = need
        elif need and fits:
            codes.add(OUT_OF_PAGES)
        counts[b] += got
        new_off.append(new_off[-1] + got)
        ok = not bad and fits and pages_of(c + t) <= counts[b]
        if served is not None:
            served.append(rows if ok else 0)
            rows = served[-1]
        q_off.append(q_off[-1] + rows)
        if ok:
            for i in range(rows):
                page = int(table[b, (c + i) // PAGE])
                if not 0 <= page < num_pages:
                    codes.add(BAD_PAGE)
                    continue
                pos[q_off[b] + i] = c + i
                slots[q_off[b] + i] = page * PAGE + (c + i) % PAGE
    return table, counts, len(stack), q_off, new_off, pos, slots, codes


def release_pages(keep, table, counts, free, free_count):
    """(counts, free, free_count, released_offsets, device codes)."""
    free = [int(p) for p in free]
    cap, n = len(free), max(0, min(int(free_count), len(free)))
    counts, off, codes = [int(c) for c in counts], [0], set()
    asked = n
    for b in range(len(keep)):
        have = counts[b]
        if not 0 <= have <= table.shape[1]:
            codes.add(BAD_LENGTH)
            off.append(off[-1])
            continue
        left = have if keep[b] < 0 else min(have, pages_of(int(keep[b])))
        asked += have - left
        if have > left and asked > cap:
            codes.add(BAD_LENGTH)
            left = have
        for j in range(left, have):
            free[n] = int(table[b][j])
            n += 1
        counts[b] = left
        off.append(off[-1] + have - left)
    return counts, free, n, off, codes


# 2 pi to 60 digits
_TURN = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def _reduced(position: int, freq: float) -> float:
    """position * freq modulo 2 pi: exact rationals, rounded once."""
    p = position * Fraction(freq)
    return float(p - (p / _TURN).__floor__() * _TURN)


def norm_rotate(x, weight, eps, inv_freq, axis, positions, interleaved, rope_scale=1.0):
    """x float64 [n, heads, D] -> normed (with a weight) and rotated, float64.
    positions: [axes, n]."""
    x = np.array(x, np.float64)
    n, heads, D = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = 0 if inv_freq is None else len(inv_freq)
    y = x.copy()
    for i in range(half):
        a = 0 if axis is None else max(0, min(int(axis[i]), len(positions) - 1))
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        for r in range(n):
            ang = _reduced(int(positions[a][r]), float(inv_freq[i]))
            c, s = math.cos(ang) * rope_scale, math.sin(ang) * rope_scale
            y[r, :, u] = x[r, :, u] * c - x[r, :, v] * s
            y[r, :, v] = x[r, :, v] * c + x[r, :, u] * s
    return y


def history(state, tokens, q_offsets, vocab, accepted=None, prompt=False, reset=False):
    """The int16 token history after a call, as int64. A sequence whose offsets are
    not usable has no tokens."""
    state = np.array(state, np.int64)
    if reset:
        state[:] = 0
    for b in range(len(q_offsets) - 1):
        end = q_offsets[b + 1]
        if not 0 <= q_offsets[b] <= end <= len(tokens):
            continue
        if accepted is not None:
            end = max(q_offsets[b], min(end, q_offsets[b] + int(accepted[b]) + 1))
        for i in range(q_offsets[b], end):
            v = int(tokens[i])
            if not 0 <= v < vocab:
                continue
            bit, n = state[b, v] < 0, int(state[b, v]) & 0x7fff
            if prompt:
                bit = True
            else:
                n = min(n + 1, 32767)
            state[b, v] = n - (32768 if bit else 0)
    return state


def choose(logits, q_offsets, tokens=None, state=None, repetition=None, presence=None,
           frequency=None, bias=None, mask=None, mask_rows=None):
    """(z5 as fp32 [n, V], choices). bias: a list of [(id, value), ...] per
    sequence. Rows of no sequence keep their logits and choice -2. numpy's fp32
    operations are correctly rounded, one rounding a step."""
    f32 = np.float32
    z_all = np.array(logits, f32)
    n, V = z_all.shape
    pick = np.full(n, -2, np.int64)
    with np.errstate(all="ignore"):
        for b in range(len(q_offsets) - 1):
            count = None
            if state is not None:
                st = np.asarray(state[b][:V], np.int64)
                count, prompt = st & 0x7fff, st < 0
                r = f32(1 if repetition is None else repetition[b])
                r = r if 0 < r < np.inf else f32(1)
                p = f32(0 if presence is None else presence[b])
                f = f32(0 if frequency is None else frequency[b])
            for row in range(q_offsets[b], q_offsets[b + 1]):
                z = z_all[row]
                if count is not None:
                    if 0 <= int(tokens[row]) < V:
                        count[int(tokens[row])] += 1
                    seen = (count > 0) | prompt
                    y = np.where(z > 0, z / r, z * r)
                    y = y - f * count.astype(f32)
                    y = np.where(count > 0, y - p, y)
                    z = np.where(seen, y, z).astype(f32)
                if bias is not None:
                    for v, x in dict(bias[b]).items():      # the last entry of an id
                        if 0 <= v < V:
                            z[v] = z[v] + f32(x)
                m = row if mask_rows is None else int(mask_rows[row])
                if mask is not None and m >= 0:
                    for v in range(V):
                        if m >= len(mask) or not (int(mask[m][v // 32]) >> (v % 32)) & 1:
                            z[v] = -np.inf
                z_all[row] = z
                left = np.where(np.isnan(z), -np.inf, z)
                pick[row] = int(np.argmax(left)) if left.max() > -np.inf else -1
    return z_all, pick


def cache_rows(pool, slots, kv_heads):
    """float64 K and V rows [n, heads, D] of the slots of an oracle pool; NaN
    rows where the slot is -1."""
    s = np.asarray(slots)
    page, at = np.maximum(s, 0) // PAGE, np.maximum(s, 0) % PAGE
    k = pool.k_codes[page, :, at].astype(np.float64) * pool.k_scales[page, :, at][..., None]
    v = pool.v_codes[page, :, at].astype(np.float64) * pool.v_scales[page, :, at][..., None]
    k[s < 0] = np.nan
    v[s < 0] = np.nan
    return k, v
