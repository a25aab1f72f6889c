"""Rows of both appends that the quantiser treats apart: zeros, zeros with NaN,
infinities, NaN among values, subnormals, and heads that do not fill a warp's rows.

The quantiser: a = max |x| (a NaN does not count), s = fl32(a / 127), code 0 where
s = 0 or the quotient is NaN, else clamp(rne(fl32(x / s)), +-127). Each step is one
correctly rounded fp32 operation, here and there: bits are compared."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def quantised(x):
    with np.errstate(all="ignore"):
        a = np.fmax.reduce(np.abs(x), axis=-1, initial=np.float32(0))
        s = (a / np.float32(127)).astype(np.float32)
        q = np.rint((x / s[..., None]).astype(np.float32))
        c = np.where(np.isnan(q) | (s == 0)[..., None], 0, np.clip(q, -127, 127))
    return c.astype(np.int8), s


def rows(seed, n, heads, D, dtype):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, heads, D)).astype(np.float32)
    kind = r.integers(0, 8, (n, heads))
    for t, h in np.ndindex(n, heads):
        row, some = x[t, h], r.random(D) < 0.2
        if kind[t, h] == 1:
            row[:] = 0
        elif kind[t, h] == 2:
            row[:] = np.where(some, np.nan, 0)
        elif kind[t, h] == 3:
            row[some] = np.inf
            row[5] = -np.inf
        elif kind[t, h] == 4:
            row[some] = np.nan
        elif kind[t, h] == 5:
            row *= np.float32(2.0 ** -130)
        elif kind[t, h] == 6:
            row[:] = np.float32(2.0 ** -149) * r.integers(-200, 200, D)
        elif kind[t, h] == 7:                        # next to (k + 1/2) steps, some exactly there
            row[:] = np.rint(row * 60) + 0.5
            row[7] = 127
    t = torch.tensor(x, device="cuda").to(dtype)
    return t, t.float().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 2, 3, 4, 5, 7, 8])
def test_both_appends(heads, D, dtype):
    n = 67
    (k, kf), (v, vf) = rows(heads, n, heads, D, dtype), rows(heads + 50, n, heads, D, dtype)
    pages = -(-n // 16)
    a, b = sk.alloc_pool(pages, heads, D), sk.alloc_pool(pages, heads, D)
    for pool in (a, b):
        for t, fill in zip(pool, (55, -55, 7.5, -7.5)):
            t.fill_(fill)
    sk.splash_kv_append(k, v, *a, i32([np.arange(pages)]), i32([0]), i32([n]))
    q = torch.zeros((n, 2 * heads, D), dtype=dtype, device="cuda")
    q_out = torch.empty_like(q, dtype=torch.bfloat16)
    sk.splash_qkv_append(q, k, v, q_out, *b, None, i32(np.arange(n)))
    for pool in (a, b):
        page, at = torch.arange(n, device="cuda") // 16, torch.arange(n, device="cuda") % 16
        for codes, scales, x in ((pool[0], pool[2], kf), (pool[1], pool[3], vf)):
            want_c, want_s = quantised(x)
            assert np.array_equal(codes[page, :, at].cpu().numpy(), want_c)
            assert np.array_equal(scales[page, :, at].cpu().numpy(), want_s)
        assert (pool[0][-1, :, n % 16:] == 55).all() and (pool[3][-1, :, n % 16:] == -7.5).all()
