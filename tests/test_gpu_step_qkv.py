"""Norm, rotation and quantised append, and cached rows by slot, on the GPU
against the fp64 oracle.

Bounds. u = 2^-24. Per value of a normed and rotated row, fp32 work is off by at
most (|a| + |b|) * 25 u for the pair (a, b) it came from: the sum of squares over
lanes and shuffles (13 u, half of it through the root), the mean and eps (2 u),
rsqrtf (4 u), two products (2 u); the angle's 2^-32 turn and its rounding to fp32
(3.2 u), sincospif (4 u), the scale and the two products of the turn (3 u). That
is below 2^-19 (|a| + |b|) (= 32 u). A bf16 output adds half a step, 2^-8 of the
value. |a| + |b| is at most twice the largest rotated value of the row, so a
scale is off by 2^-18 of itself and value / scale by 127 * 3 * 2^-18 < 2e-3
steps: a code differs only where the oracle's quotient is within 2e-3 of a half,
and then by one.
"""
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

from oracle import splash_oracle as O  # noqa: E402
from oracle import step_oracle as S  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make(seed, n, hq, hkv, D, dtype, pages=None, layout="packed", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, hq + 2 * hkv, D), generator=g, device="cuda") * scale
    x[:, :, 3] *= 8
    x = x.to(dtype)
    if layout == "packed":
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    elif layout == "separate":
        q, k, v = (t.contiguous() for t in (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]))
    else:                    # heads first, each head's rows with a gate beside them
        y = torch.zeros((hq + 2 * hkv, n, 2 * D), dtype=dtype, device="cuda")
        y[:, :, :D] = x.transpose(0, 1)
        z = y[:, :, :D].transpose(0, 1)
        q, k, v = z[:, :hq], z[:, hq:hq + hkv], z[:, hq + hkv:]
    pages = pages or -(-n // 16) + 2
    slots = torch.randperm(pages * 16, generator=g, device="cuda")[:n].int()
    return q, k, v, slots, pages


def pool_of(pages, hkv, D):
    """A pool whose unwritten bytes would show."""
    p = sk.alloc_pool(pages, hkv, D)
    p[0].fill_(55)
    p[1].fill_(-55)
    p[2].fill_(7.5)
    p[3].fill_(-7.5)
    return p


def run(q, k, v, slots, pages, pos=None, q_out=None, **kw):
    hkv, D = k.shape[1], k.shape[2]
    pool = pool_of(pages, hkv, D)
    q_out = torch.full(q.shape, 99.0, dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.splash_qkv_append(q, k, v, q_out, *pool, pos, slots, device_status=st, **kw)
    torch.cuda.synchronize()
    return q_out, pool, st.item()


def cached(pool, slots):
    page, at = slots.long() // 16, slots.long() % 16
    return [pool[0][page, :, at].cpu().numpy(), pool[1][page, :, at].cpu().numpy(),
            pool[2][page, :, at].cpu().numpy(), pool[3][page, :, at].cpu().numpy()]


def f64(t):
    return t.double().cpu().numpy()


def check_q(q_out, want):
    got = f64(q_out)
    pair = 2 * np.abs(want).max(-1, keepdims=True)
    off = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -19 * pair)
    assert np.isfinite(got).all() and off.max() <= 0, off.max()


def check_codes(codes, scales, want):
    a = np.abs(want).max(-1)
    assert (np.abs(scales - a / 127) <= a / 127 * (2.0 ** -18 + 2.0 ** -23)).all()
    ratio = np.divide(want, (a / 127)[..., None], out=np.zeros_like(want), where=a[..., None] > 0)
    near = np.abs(np.abs(ratio - np.trunc(ratio)) - 0.5) < 2e-3
    d = np.abs(codes - np.clip(np.rint(ratio), -127, 127))
    assert (d[~near] == 0).all() and d.max(initial=0) <= 1


def check_exact(codes, scales, x):
    want_c, want_s = O.quantise_rows(x.reshape(-1, x.shape[-1]))
    assert np.array_equal(codes.reshape(-1, x.shape[-1]), want_c)
    assert np.array_equal(scales.reshape(-1), want_s)


def untouched(pool, slots, pages):
    free = torch.ones(pages * 16, dtype=torch.bool, device="cuda")
    free[slots.long().clamp(min=0)[slots >= 0]] = False
    m = free.view(pages, 1, 16).expand(-1, pool[0].shape[1], -1)
    assert (pool[0][m] == 55).all() and (pool[1][m] == -55).all()
    assert (pool[2][m] == 7.5).all() and (pool[3][m] == -7.5).all()


def freqs(half, base=1e4):
    return torch.tensor(base ** (-np.arange(half) / max(half, 1)), dtype=torch.float32, device="cuda")


# (tokens, q heads, KV heads): one row, heads that do not fill a warp's groups,
# more head rows than are in flight, tokens enough for a warp each
SHAPES = [(1, 1, 1), (3, 7, 1), (5, 12, 3), (33, 24, 4), (2, 40, 20), (700, 8, 2), (6000, 2, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm_and_rotation(shape, D, dtype):
    n, hq, hkv = shape
    big = n >= 700
    q, k, v, slots, pages = make(n + D, n, hq, hkv, D, dtype)
    r = np.random.default_rng(n)
    pos = r.integers(0, 131072, (1, n))
    w = [torch.tensor(r.uniform(0.5, 1.5, D), dtype=torch.float32, device="cuda") for _ in range(2)]
    for rot, paired in ((D, False), (D // 2, True)) if not big else ((D, bool(D == 128)),):
        f = freqs(rot // 2)
        q_out, pool, st = run(q, k, v, slots, pages, i32(pos[0]), inv_freq=f, q_weight=w[0],
                              k_weight=w[1], interleaved=paired)
        assert st == 0
        pick = np.arange(n) if not big else r.choice(n, 40, replace=False)
        ff = f64(f)
        kc, vc, ks, vs = cached(pool, slots)
        check_q(q_out[pick.tolist()], S.norm_rotate(f64(q)[pick], f64(w[0]), 1e-6, ff, None,
                                                    pos[:, pick], paired))
        check_codes(kc[pick], ks[pick], S.norm_rotate(f64(k)[pick], f64(w[1]), 1e-6, ff, None,
                                                      pos[:, pick], paired))
        check_exact(vc[pick], vs[pick], v.float().cpu().numpy()[pick])
        untouched(pool, slots, pages)


@pytest.mark.parametrize("layout", ["packed", "separate", "gated"])
@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 128])
@pytest.mark.parametrize("paired", [False, True])
def test_partial_rotations_and_layouts(rot, paired, layout):
    n, hq, hkv, D = 9, 5, 2, 128
    for dtype in (torch.float32, torch.bfloat16):
        q, k, v, slots, pages = make(rot, n, hq, hkv, D, dtype, layout=layout)
        pos = np.arange(n)[None] * 977
        f = freqs(rot // 2)
        q_out, pool, st = run(q, k, v, slots, pages, i32(pos[0]), inv_freq=f, interleaved=paired)
        assert st == 0
        kc, vc, ks, vs = cached(pool, slots)
        wq = S.norm_rotate(f64(q), None, 0, f64(f), None, pos, paired)
        check_q(q_out, wq)
        if rot == 0:              # nothing but the quantiser: bit for bit
            assert torch.equal(q_out, q.to(torch.bfloat16))
            check_exact(kc, ks, k.float().cpu().numpy())
        else:
            check_codes(kc, ks, S.norm_rotate(f64(k), None, 0, f64(f), None, pos, paired))
            # the values past the rotated ones are only rounded
            assert torch.equal(q_out[..., rot:], q[..., rot:].to(torch.bfloat16))
        check_exact(vc, vs, v.float().cpu().numpy())


def test_one_norm_alone():
    n, hq, hkv, D = 4, 3, 2, 256
    q, k, v, slots, pages = make(1, n, hq, hkv, D, torch.bfloat16)
    w = torch.rand(D, device="cuda") + 0.5
    q_out, pool, _ = run(q, k, v, slots, pages, q_weight=w, eps=1e-5)
    check_q(q_out, S.norm_rotate(f64(q), f64(w), 1e-5, None, None, None, False))
    check_exact(cached(pool, slots)[0], cached(pool, slots)[2], k.float().cpu().numpy())
    q_out, pool, _ = run(q, k, v, slots, pages, k_weight=w, eps=1e-5)
    assert torch.equal(q_out, q)
    c = cached(pool, slots)
    check_codes(c[0], c[2], S.norm_rotate(f64(k), f64(w), 1e-5, None, None, None, False))


@pytest.mark.parametrize("axes,axis_of", [
    (3, lambda i, h: i * 3 // h), (3, lambda i, h: i % 3), (2, lambda i, h: i % 2),
    (3, lambda i, h: [7, -2, 1][i % 3]),                # cut to the axes there are
    (3, None),                                          # no table: axis 0
])
@pytest.mark.parametrize("paired", [False, True])
def test_several_axes(axes, axis_of, paired):
    n, hq, hkv, D = 7, 4, 1, 128
    q, k, v, slots, pages = make(axes, n, hq, hkv, D, torch.bfloat16)
    pos = np.random.default_rng(axes).integers(0, 5000, (axes, n))
    f = freqs(32)
    ax = None if axis_of is None else [axis_of(i, 32) for i in range(32)]
    q_out, pool, st = run(q, k, v, slots, pages, i32(pos), inv_freq=f, interleaved=paired,
                          freq_axis=None if ax is None else i32(ax), rope_scale=1.25)
    assert st == 0
    check_q(q_out, S.norm_rotate(f64(q), None, 0, f64(f), ax, pos, paired, 1.25))
    c = cached(pool, slots)
    check_codes(c[0], c[2], S.norm_rotate(f64(k), None, 0, f64(f), ax, pos, paired, 1.25))


def test_far_positions_and_odd_frequencies():
    """Angles stay exact to the end of the 32-bit range, for frequencies of any
    size and sign."""
    pos = np.array([[0, 1, 131071, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -5, 99]])
    n, hq, hkv, D = pos.shape[1], 2, 1, 64
    q, k, v, slots, pages = make(3, n, hq, hkv, D, torch.float32)
    f = torch.tensor([1.0, 0.7071, 1e-3, 1e-9, 1e-30, 1e-42, 0.0, -0.3, 2.5, 100.0, 6.2831853,
                      1e-4, 3e-7, 0.1, 0.9999, 1e-5], dtype=torch.float32, device="cuda")
    q_out, pool, st = run(q, k, v, slots, pages, i32(pos[0]), inv_freq=f)
    assert st == 0
    want = S.norm_rotate(f64(q), None, 0, f64(f), None, pos, False)
    check_q(q_out, want)


def test_padded_rows_and_bad_slots_write_nothing():
    n, hq, hkv, D = 20, 4, 2, 128
    q, k, v, slots, pages = make(8, n, hq, hkv, D, torch.bfloat16)
    slots[3] = -1
    slots[15:] = -1
    q_out, pool, st = run(q, k, v, slots, pages, i32(np.arange(n)), inv_freq=freqs(64))
    assert st == 0
    dead = (slots < 0).cpu()
    assert (q_out[dead] == 99).all() and (q_out[~dead] != 99).any()
    untouched(pool, slots, pages)
    slots[5] = pages * 16
    q_out, pool, st = run(q, k, v, slots, pages, i32(np.arange(n)), inv_freq=freqs(64))
    assert st == sk.DEVICE_BAD_PAGE and (q_out[5] == 99).all() and (q_out[4] != 99).any()
    slots[5] = -1
    untouched(pool, slots, pages)


def test_zero_and_extreme_rows():
    n, hq, hkv, D = 6, 2, 2, 64
    x = np.random.default_rng(2).standard_normal((n, 6, D)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e15
    x[3, :, 1:] = 0
    x[4] = 2.0 ** -140                      # subnormal
    t = torch.tensor(x, device="cuda")
    slots, pages = i32(np.arange(n)), 1
    q_out, pool, _ = run(t[:, :2], t[:, 2:4], t[:, 4:], slots, pages)
    c = cached(pool, slots)
    check_exact(c[0], c[2], x[:, 2:4])
    check_exact(c[1], c[3], x[:, 4:])
    w = torch.ones(D, device="cuda")
    q_out, pool, _ = run(t[:, :2], t[:, 2:4], t[:, 4:], slots, pages, q_weight=w, k_weight=w)
    check_q(q_out[:4], S.norm_rotate(x[:4, :2], np.ones(D), 1e-6, None, None, None, False))
    assert (q_out[0] == 0).all() and (cached(pool, slots)[0][0] == 0).all()


def test_the_append_agrees_with_kv_append():
    """Without norm and rotation the cache holds what splash_kv_append writes."""
    n, hkv, D = 37, 4, 256
    q, k, v, _, _ = make(4, n, 8, hkv, D, torch.bfloat16, layout="separate")
    table, ctx, T = i32([[2, 0, 3, 1]]), i32([5]), i32([n])
    old = pool_of(4, hkv, D)
    sk.splash_kv_append(k, v, *old, table, ctx, T)
    p = np.arange(5, 5 + n)
    slots = i32(np.array([2, 0, 3, 1])[p // 16] * 16 + p % 16)
    _, new, _ = run(q, k, v, slots, 4)
    assert all(torch.equal(a, b) for a, b in zip(old, new))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_next_to_rounding_borders(D):
    """Values within a few ulps of (k + 1/2) steps, for scales of many sizes: the
    codes of both appends are those of the division, bit for bit."""
    r = np.random.default_rng(D)
    n, hkv = 64, 2
    a = np.exp2(r.uniform(-120, 120, (n, hkv, 1))).astype(np.float32)
    a[:8] = np.exp2(r.integers(-149, -120, (8, hkv, 1))).astype(np.float32)      # subnormal steps
    s = (a / np.float32(127)).astype(np.float32)
    k = r.integers(-127, 127, (n, hkv, D)) + 0.5
    x = (k * s.astype(np.float64)).astype(np.float32)
    ulps = r.integers(-3, 4, x.shape).astype(np.int32)
    x = np.where(x == 0, x, (x.view(np.int32) + ulps).view(np.float32))
    x = np.clip(x, -a, a)
    x[:, :, 5] = a[:, :, 0]
    t = torch.tensor(x, device="cuda")
    q_out, pool, _ = run(t[:, :1].contiguous(), t, -t, i32(np.arange(n)), n // 16)
    c = cached(pool, i32(np.arange(n)))
    check_exact(c[0], c[2], x)
    check_exact(c[1], c[3], -x)
    old = pool_of(n // 16, hkv, D)
    sk.splash_kv_append(t, -t, *old, i32([np.arange(n // 16)]), i32([0]), i32([n]))
    assert all(torch.equal(a, b) for a, b in zip(old, pool))


def test_q_in_place_and_on_another_stream():
    n, hq, hkv, D = 50, 8, 2, 128
    q, k, v, slots, pages = make(6, n, hq, hkv, D, torch.bfloat16, layout="separate")
    pos, f, w = i32(np.arange(n) * 31), freqs(64), torch.rand(D, device="cuda") + 0.5
    want, pool, _ = run(q, k, v, slots, pages, pos, inv_freq=f, q_weight=w)
    own = q.clone()
    run(own, k, v, slots, pages, pos, q_out=own, inv_freq=f, q_weight=w)
    assert torch.equal(own, want)
    s = torch.cuda.Stream()
    out, p2 = torch.zeros_like(want), pool_of(pages, hkv, D)
    torch.cuda.synchronize()
    sk.splash_qkv_append(q, k, v, out, *p2, pos, slots, inv_freq=f, q_weight=w, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(pool, p2))


def test_a_captured_append_follows_its_inputs():
    n, hq, hkv, D = 12, 8, 2, 128
    q, k, v, slots, pages = make(7, n, hq, hkv, D, torch.bfloat16, layout="separate")
    pos, f = i32(np.arange(n)), freqs(64)
    out, pool = torch.zeros_like(q), pool_of(pages, hkv, D)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.splash_qkv_append(q, k, v, out, *pool, pos, slots, inv_freq=f)
    for add in (0, 1000):
        pos.add_(add)
        q.mul_(0.5)
        g.replay()
        want, wpool, _ = run(q, k, v, slots, pages, pos, inv_freq=f)
        assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(pool, wpool))


def test_a_pool_past_4_gib():
    """Code offsets past 32 bits: 2^21 pages x 1 head x 2 * 16 * 64 = 4.3 GB."""
    pages, hkv, D, n = 2 ** 21 + 4, 1, 64, 5
    pool = sk.alloc_pool(pages, hkv, D)
    q, k, v, _, _ = make(9, n, 1, hkv, D, torch.bfloat16)
    last = pages * 16 - 1
    slots = i32([0, last, last - 16, 2 ** 25, 2 ** 25 + 17])
    out = torch.empty((n, 1, D), dtype=torch.bfloat16, device="cuda")
    sk.splash_qkv_append(q, k, v, out, *pool, None, slots)
    kb, vb = (torch.zeros((n, hkv, D), device="cuda") for _ in range(2))
    sk.splash_kv_gather(*pool, slots, kb, vb)
    torch.cuda.synchronize()
    kc, vc, ks, vs = cached(pool, slots)
    check_exact(kc, ks, k.float().cpu().numpy())
    check_exact(vc, vs, v.float().cpu().numpy())
    assert np.array_equal(kb.cpu().numpy(), kc.astype(np.float32) * ks[..., None])
    assert np.array_equal(vb.cpu().numpy(), vc.astype(np.float32) * vs[..., None])


# ---------------------------------------------------------------------------
# gather
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,hkv,D", [(1, 1, 64), (5, 3, 64), (77, 2, 128), (400, 5, 256),
                                     (9000, 4, 256), (20000, 1, 64)])
def test_gather_rows(n, hkv, D, dtype):
    pages = -(-n // 16) + 3
    g = torch.Generator(device="cuda").manual_seed(n)
    pool = sk.alloc_pool(pages, hkv, D)
    for t in pool[:2]:
        t.copy_(torch.randint(-127, 128, t.shape, generator=g, device="cuda", dtype=torch.int8))
    for t in pool[2:]:
        t.copy_(torch.rand(t.shape, generator=g, device="cuda") + 0.01)
    slots = torch.randint(0, pages * 16, (n,), generator=g, device="cuda").int()   # some twice
    slots[::7] = -1
    k, v = (torch.full((n, hkv, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.splash_kv_gather(*pool, slots, k, v, device_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    page, at = slots.long().clamp(min=0) // 16, slots.long().clamp(min=0) % 16
    live = (slots >= 0)[:, None, None]
    for got, c, s in ((k, pool[0], pool[2]), (v, pool[1], pool[3])):
        want = (c[page, :, at].float() * s[page, :, at][..., None]).to(dtype)
        assert torch.equal(got, torch.where(live, want, torch.full_like(want, 3.0)))
    slots[0] = pages * 16
    sk.splash_kv_gather(*pool, slots, k, v, device_status=st)
    assert st.item() == sk.DEVICE_BAD_PAGE and (k[0] == 3).all()


def test_no_rows_is_no_work():
    pool = sk.alloc_pool(2, 1, 64)
    before = sk.splash_launch_count()
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    sk.splash_kv_gather(*pool, i32([]), e, e.clone())
    sk.splash_qkv_append(e, e, e, e.clone(), *pool, None, i32([]))
    assert sk.splash_launch_count() == before


def test_rows_further_apart_than_32_bits():
    """Token strides past 2^31 values."""
    n, far, D = 3, 2 ** 31 + 64, 128
    q, k, v, slots, pages = make(10, n, 4, 1, D, torch.bfloat16)
    wide = torch.empty(2 * far + 6 * D, dtype=torch.bfloat16, device="cuda")
    row = wide.as_strided((n, 6, D), (far, D, 1))
    row[:, :4], row[:, 4:5], row[:, 5:] = q, k, v
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    f = torch.rand(D // 2, device="cuda")
    want, wpool, _ = run(q, k, v, slots, pages, pos, inv_freq=f)
    got, gpool, _ = run(row[:, :4], row[:, 4:5], row[:, 5:], slots, pages, pos, inv_freq=f)
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(gpool, wpool))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,hq,hkv", [(3, 20, 6), (700, 24, 4), (2431, 3, 1), (5003, 5, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_token_comes_out_the_same_in_a_call_of_many_and_of_few(n, hq, hkv, D, dtype):
    """A warp's tokens, with skipped ones between, against calls of 1 to 40 tokens,
    where every batch of a token has a warp of its own."""
    q, k, v, slots, pages = make(n + hq, n, hq, hkv, D, dtype)
    g = torch.Generator(device="cuda").manual_seed(n)
    slots[torch.rand(n, generator=g, device="cuda") < 0.4] = -1
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    f = torch.rand(D // 2, generator=g, device="cuda")
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    a = dict(inv_freq=f, q_weight=w, k_weight=w)
    want, wpool, st = run(q, k, v, slots, pages, pos, **a)
    got, gpool = torch.full_like(want, 99.0), pool_of(pages, hkv, D)
    at = 0
    while at < n:
        m = min(n - at, 1 + at % 40)
        part = slice(at, at + m)
        sk.splash_qkv_append(q[part], k[part], v[part], got[part], *gpool, pos[part], slots[part], **a)
        at += m
    assert st == 0 and torch.equal(got, want)
    assert all(torch.equal(x, y) for x, y in zip(gpool, wpool))
