"""Log probabilities, entropy and alternatives on the GPU against 64 bits.

Bounds (u = 2^-24). The maximum is exact. An exponent's argument t = (z - m) log2 e
comes out of one fused product of fp32 values with |z log2 e|, |m log2 e| <= A:
off by 2 u A + u |t|; ex2 by 2^-22. Weights therefore by w = ln 2 (3 u A) + 2^-22 of
themselves, and S by that and its additions: values are added 2 to a pair and at most
L = (values of a lane) in a row, then over a few levels, L u + 10 u in all, with L
at most 1024 here. Moving the reference adds 2^-22 a move, at most 16 here.
  log p: w + (L + 10) u + 2^-18 + 4 u (|log p| + ln S)
  entropy: (2 w + 2 (L + 10) u + 2^-17) (1 + sum p |ln p|), since its terms are p times
  |t| <= |ln p| + ln S / ...: bounded with the same factor by 1 + H + ln V.
"""
from __future__ import annotations

import math
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

U = 2.0 ** -24
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def i32(a):
    return torch.tensor(np.asarray(a), device="cuda").to(torch.int32)


def run(z, tokens, k, rows=None, **over):
    m = z.shape[0] if rows is None else len(rows)
    o = dict(logprobs=torch.full((m,), 5.0, device="cuda"),
             entropy=torch.full((m,), 5.0, device="cuda"),
             top_ids=torch.full((m, k), 5, dtype=torch.int32, device="cuda") if k else None,
             top_logprobs=torch.full((m, k), 5.0, device="cuda") if k else None)
    o.update(over)
    status = i32([0])
    ws = sk.alloc_logprobs_workspace(m, z.shape[1])
    ws.fill_(0xff)
    sk.splash_token_logprobs(z, ws, tokens=None if o["logprobs"] is None else i32(tokens),
                             rows=None if rows is None else i32(rows), device_status=status, **o)
    torch.cuda.synchronize()
    return o, status.item()


def want_of(z, tokens, k):
    """The oracle's values, by torch in 64 bits for rows that it would take long on."""
    z64 = z.double().cpu().numpy()
    if z64.shape[1] <= 2000:
        return T.logprobs(z64, tokens, k)
    z64 = np.where(np.isnan(z64), -np.inf, z64)
    lp, ent, ids, tops = [], [], [], []
    for x, t in zip(z64, tokens):
        p = x - x.max()
        p = p - np.log(np.exp(p).sum())
        live = p > -np.inf
        order = np.argsort(-x, kind="stable")[:k]
        lp.append(p[t])
        ent.append(-(np.exp(p[live]) * p[live]).sum())
        ids.append(np.where(x[order] > -np.inf, order, -1))
        tops.append(p[order])
    return np.array(lp), np.array(ent), np.array(ids).reshape(len(lp), k), np.array(tops).reshape(len(lp), k)


def check(z, tokens, o, k, at=None):
    lp, ent, ids, tops = want_of(z, tokens, k)
    at = range(len(lp)) if at is None else at
    z64 = z.double().cpu().numpy()
    for i, r in enumerate(at):
        if r is None:
            continue
        live = z64[r][np.isfinite(z64[r])]
        A = 1.4427 * (np.abs(live).max() if len(live) else 0)
        w = 0.7 * 3 * U * A + 2.0 ** -22
        near = lambda x: w + 1034 * U + 2.0 ** -18 + 4 * U * (abs(x) + math.log(z.shape[1]))  # noqa: E731
        got = o["logprobs"][i].item()
        assert got == lp[r] if lp[r] == -np.inf else abs(got - lp[r]) <= near(lp[r]), (r, got, lp[r])
        e = o["entropy"][i].item()
        bound = (2 * w + 2 * 1034 * U + 2.0 ** -17) * (1 + ent[r] + math.log(z.shape[1]))
        assert e >= 0 and abs(e - ent[r]) <= bound, (r, e, ent[r])
        if k:
            assert o["top_ids"][i].tolist() == ids[r].tolist(), r
            for g, x in zip(o["top_logprobs"][i].tolist(), tops[r]):
                assert g == x if x == -np.inf else abs(g - x) <= near(x), (r, g, x)


def make(seed, n, V, kind, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (spread * torch.randn((n, V), generator=g, device="cuda")).to(KINDS[kind])
    return z, torch.randint(0, V, (n,), generator=g, device="cuda").tolist()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 511, 512, 513, 1000, 1025, 1999])
@pytest.mark.parametrize("k", [0, 1, 5, 32])
def test_small_vocabularies(kind, V, k):
    z, tokens = make(V + k, 5, V, kind)
    o, st = run(z, tokens, k)
    assert st == 0
    check(z, tokens, o, k)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("V,n", [(32768, 1), (100003, 3), (131072, 2), (262145, 2), (300001, 1),
                                 (5003, 400)])
def test_large_vocabularies(kind, V, n):
    z, tokens = make(V, n, V, kind)
    o, st = run(z, tokens, 20)
    assert st == 0
    check(z, tokens, o, 20)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 5, 7])
def test_any_alignment_and_stride(kind, shift):
    z, tokens = make(shift, 6, 1291, kind)
    wide = torch.full((6, 1291 + 40 + shift), 300.0, dtype=z.dtype, device="cuda")
    view = wide[:, shift:shift + 1291]                 # what lies beside the rows is larger
    view.copy_(z)
    o, _ = run(view, tokens, 9)
    check(z, tokens, o, 9)


@pytest.mark.parametrize("kind", list(KINDS))
def test_masked_values_and_the_ends_of_the_range(kind):
    low, high = torch.finfo(KINDS[kind]).min, torch.finfo(KINDS[kind]).max
    n, V = 14, 1100
    z, tokens = make(1, n, V, kind)
    inf = math.inf
    z[0] = -inf
    z[1, ::2] = -inf
    z[2, 3:] = -inf                                    # fewer than are asked for
    z[3] = low                                         # the type's lowest as a mask: all alike
    z[4, 5:] = low
    z[5, :1000], z[5, 1000:] = -inf, low
    z[6, ::3] = math.nan
    z[7] = math.nan
    z[8, 17] = inf
    z[9, 100:104], z[9, 600] = inf, high
    z[10] = high
    z[11, 1:] = low / 2
    z[11, 0] = low
    z[12, ::2], z[12, 1::2] = 0.0, -0.0                # equal: the lowest index first
    z[13, 700:] = z[13, 700:] * 0 - 500
    tokens[2], tokens[5], tokens[8], tokens[9], tokens[6] = 900, 1050, 17, 600, 3
    o, st = run(z, tokens, 8)
    assert st == 0
    check(z, tokens, o, 8)


@pytest.mark.parametrize("kind", list(KINDS))
def test_equal_values_by_index(kind):
    """Few different values: more equal ones at the border than any list holds."""
    g = torch.Generator(device="cuda").manual_seed(4)
    z = torch.randint(0, 3, (4, 40000), generator=g, device="cuda").to(KINDS[kind])
    z[1] = 1
    z[2, :39000] = 0
    z[3, -1] = 5
    o, _ = run(z, [0, 1, 2, 3], 32)
    check(z, [0, 1, 2, 3], o, 32)


def test_growing_rows_move_the_reference():
    z = torch.linspace(-900, 900, 8192, device="cuda").repeat(3, 1)
    z[1] = z[1].flip(0)
    z[2] = torch.linspace(-8, 8, 8192, device="cuda")
    tokens = [8191, 0, 4000]
    o, _ = run(z, tokens, 4)
    check(z, tokens, o, 4)


def test_row_lists():
    z, tokens = make(9, 12, 3001, "bf16")
    rows = [3, -1, 3, 11, 0, -5, 7]
    o, st = run(z, tokens, 3, rows=rows)
    assert st == 0
    check(z, tokens, o, 3, at=[r if r >= 0 else None for r in rows])
    want, _ = run(z, tokens, 3)
    for i, r in enumerate(rows):
        for name, t in o.items():
            assert torch.equal(t[i], want[name][r]) if r >= 0 else (t[i] == 5).all()
    o, st = run(z, tokens, 3, rows=[2, 12, 1])
    assert st == sk.DEVICE_BAD_LENGTH and o["logprobs"][1] == 5
    check(z, tokens, o, 3, at=[2, None, 1])


def test_tokens_outside_the_vocabulary_and_outputs_left_out():
    z, tokens = make(10, 4, 1001, "fp32")
    full, _ = run(z, tokens, 6)
    o, st = run(z, [-1, 1001, 2 ** 31 - 1, 5], 6)
    assert st == 0 and o["logprobs"][:3].tolist() == [-math.inf] * 3
    assert torch.equal(o["top_ids"], full["top_ids"]) and torch.equal(o["entropy"], full["entropy"])
    o, _ = run(z, tokens, 0)
    assert torch.equal(o["logprobs"], full["logprobs"])
    o, _ = run(z, tokens, 6, logprobs=None)
    assert torch.equal(o["top_logprobs"], full["top_logprobs"])
    o, _ = run(z, tokens, 6, entropy=None)
    assert torch.equal(o["logprobs"], full["logprobs"])


def test_the_same_call_is_bitwise_the_same_and_streams_and_graphs():
    z, tokens = make(11, 37, 50257, "bf16")
    a, _ = run(z, tokens, 20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, _ = run(z, tokens, 20)
    o = {k: torch.zeros_like(v) for k, v in a.items()}
    ws, tok = sk.alloc_logprobs_workspace(37, 50257), i32(tokens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.splash_token_logprobs(z, ws, tokens=tok, **o)
    g.replay()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], o[k])


def test_rows_more_than_two_gigabytes_apart():
    z = torch.zeros((3, 1 << 30), dtype=torch.bfloat16, device="cuda")[:, :4000]
    z.copy_(make(12, 3, 4000, "bf16")[0])
    o, _ = run(z, [1, 2, 3], 5)
    check(z, [1, 2, 3], o, 5)
