"""Log probabilities of rows whose logits are large, or hold finite values as masks.

Bounds (u = 2^-24), from distances to the maximum, so that neither masked fills nor an
offset common to a row widens them. A weight's exponent t = (z - m) log2 e is one fused
product and a correction of its reference, fp32: off by 2 u |t| + 2 u |t| (the constant)
+ 2^-22 (the correction's own rounding); the exponential by 2^-22. A weight p is then off
by p (2^-21 + 4 u |ln p - ln p_max|), and S by S (2^-21 + 4 u D), D = sum p |ln p - ln
p_max|. A lane adds at most 8 blocks * 16 pairs = 128 values in a row, the lanes and runs
10 levels more: 138 u. A reference moves at most 8 times a run: 8 * 2^-22, and once where
runs are joined. Together r = 138 u + 2^-18 + 4 u D.
  log p: r + 4 u (|log p| + ln S), and never above 0
  entropy: r (1 + H + D) + 4 u (ln S + H)  (each term p |t| is off by r of itself)
A row of V equal values has V weights alike: log p = -ln V and H = ln V, to r with D = 0.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_logprobs import KINDS, U, make, run, want_of  # noqa: E402

K = 6


def near(z, tokens, o, rows=None):
    lp, ent, ids, tops = want_of(z, tokens, K)
    z64 = np.nan_to_num(z.double().cpu().numpy(), nan=-np.inf)
    for i in range(len(z64)) if rows is None else rows:
        x = z64[i] - z64[i].max()
        p = np.exp(x)
        S = p.sum()
        live = p > 0
        D = float(-(p[live] * x[live]).sum() / S)
        r = 138 * U + 2.0 ** -18 + 4 * U * D
        for got, want in [(o["logprobs"][i].item(), lp[i])] + list(zip(o["top_logprobs"][i].tolist(),
                                                                      tops[i])):
            assert got <= 0, (i, got)
            assert got == want if want == -np.inf else \
                abs(got - want) <= r + 4 * U * (abs(want) + math.log(S)), (i, got, want)
        e = o["entropy"][i].item()
        assert e >= 0 and abs(e - ent[i]) <= r * (1 + ent[i] + D) + 4 * U * (math.log(S) + ent[i]), \
            (i, e, ent[i])
        assert o["top_ids"][i].tolist() == ids[i].tolist(), i


FILLS = {"fp32": [-1e4, -1e6, -1e9, -1e10, -1e20, -1e30, -1e36, -3e38],
         "bf16": [-1e4, -1e6, -1e9, -1e10, -1e20, -1e30, -1e36, -3e38],
         "fp16": [-100, -1e4, -3e4, -6.5e4]}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("V", [1100, 40003])
def test_finite_fills_over_whole_blocks_and_runs(kind, V):
    """A mask's fill at the start, in the middle, at the end, in every second value, and
    everywhere but one value."""
    for fill in FILLS[kind]:
        z, tokens = make(V, 6, V, kind)
        z[0, :V // 2] = fill
        z[1, V // 3:V // 3 * 2] = fill
        z[2, V // 2:] = fill
        z[3, ::2] = fill
        z[4, :V // 2], z[4, V // 2 + 1:] = fill, fill
        z[5, 1:] = fill
        tokens[0], tokens[4], tokens[5] = 7, V // 2, 0
        o, st = run(z, tokens, K)
        assert st == 0
        near(z, tokens, o)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("V", [512, 1025, 65536])
def test_rows_of_one_value_alone(kind, V):
    values = [0.0, 3.0, -60.5, 60.5, 1e3, -3e4, 6e4]
    values += [] if kind == "fp16" else [1e6, -1e9, 1e10, -1e10, 1e20, -1e30, 1e36, -1e36, 1e38, -3e38]
    z = torch.tensor(values, device="cuda").to(KINDS[kind])[:, None].repeat(1, V)
    tokens = [V - 1] * len(values)
    o, st = run(z, tokens, K)
    assert st == 0
    for name, want in (("logprobs", -math.log(V)), ("top_logprobs", -math.log(V)),
                       ("entropy", math.log(V))):
        assert (o[name].double() - want).abs().max().item() <= 138 * U + 2.0 ** -18 + 8 * U * math.log(V), name
    assert o["top_ids"].tolist() == [list(range(K))] * len(values)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("offset", [60.5, -60.5, 1e3, 2e4, -6e4, 1e6, -1e6, 1e9])
def test_an_offset_common_to_the_row(kind, offset):
    if kind == "fp16" and abs(offset) > 65000:
        pytest.skip("past the type's range")
    z, tokens = make(3, 5, 9001, "fp32")
    step = max(abs(offset) * torch.finfo(KINDS[kind]).eps, 1e-3)       # several values a step
    z = ((z * step).double() + offset).to(KINDS[kind])
    o, st = run(z, tokens, K)
    assert st == 0
    near(z, tokens, o)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("top", [0.3, 17.3, 60.5, 3e4, 1e30])
def test_a_token_that_holds_all_the_weight(kind, top):
    """ln p is 0 and not above it, wherever the value stands and whatever came before."""
    if kind == "fp16" and top > 65000:
        pytest.skip("past the type's range")
    V = 20000
    z = torch.full((4, V), top / 2 - 200, device="cuda").to(KINDS[kind])
    tokens = [0, V - 1, 9999, 4097]
    for r, t in enumerate(tokens):
        z[r, t] = top
    z[3, :4097] = torch.linspace(top / 2 - 200, top - 40, 4097, device="cuda").to(KINDS[kind])
    o, _ = run(z, tokens, K)
    near(z, tokens, o)
    # (40 below 1e30, or below 30000 in bf16, is the same value: such rows have several)
    alone = [r for r in range(4) if (z[r] == z[r].max()).sum().item() == 1]
    assert len(alone) >= 3
    assert o["logprobs"][alone].abs().max().item() <= 2.0 ** -20
    assert o["entropy"][alone].max().item() <= 2.0 ** -18


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_large_values_of_both_signs(kind):
    """Distances between values that pass the range of an exponent, or of the type."""
    z, tokens = make(5, 6, 5000, kind)
    for r, size in enumerate([1e3, 1e5, 1e10, 1e25, 1e37, 5e37]):
        z[r] = (z[r].double() * size / 3).to(KINDS[kind])
        tokens[r] = int(z[r].argmax())
    o, st = run(z, tokens, K)
    assert st == 0
    near(z, tokens, o)


@pytest.mark.parametrize("V", [24, 600, 40000])
@pytest.mark.parametrize("k", [2, 5, 32])
def test_infinity_and_the_largest_finite_value_are_equal(V, k):
    """The lowest index first, wherever the two stand; every one of them has ln p = -ln 4."""
    z = torch.randn((2, V), generator=torch.Generator(device="cuda").manual_seed(V), device="cuda")
    big, inf = torch.finfo(torch.float32).max, math.inf
    z[0, 3], z[0, 10], z[0, 17], z[0, V - 1] = big, inf, big, inf
    z[1, 3], z[1, 10], z[1, 17], z[1, V - 1] = inf, big, inf, big
    o, st = run(z, [17, 17], k)
    assert st == 0
    for r in range(2):
        assert o["top_ids"][r].tolist()[:4] == [3, 10, 17, V - 1][:k]
    near4 = lambda x: (x.double() + math.log(4)).abs().max().item() <= 2.0 ** -18  # noqa: E731
    assert near4(o["logprobs"]) and near4(o["top_logprobs"][:, :4])
    assert near4(-o["entropy"])
