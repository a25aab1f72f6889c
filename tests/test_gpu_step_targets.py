"""Target choices and the token history on the GPU against the step oracle.

Every step of a processed logit is one correctly rounded fp32 operation on both
sides, so processed logits and choices are compared for equality."""
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

from oracle import step_oracle as S  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f32(a):
    return torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")


class Scene:
    """Logits, histories, biases and masks of one batch."""

    def __init__(self, seed, T, V, kind, stride=None, start=0, masks="all", nbias=5, tail=0,
                 dense_state=0.05):
        r = np.random.default_rng(seed)
        self.r, self.T, self.V = r, T, V
        self.q = np.concatenate([[0], np.cumsum(T)]).astype(int)
        n = int(self.q[-1]) + tail
        self.n, B = n, len(T)
        stride = V if stride is None else stride
        flat = torch.zeros(start + n * stride + 8, dtype=KINDS[kind], device="cuda")
        self.logits = flat[start:start + n * stride].view(n, stride)[:, :V]
        # a few distinct values, so that ties are many
        self.logits.copy_(torch.tensor(np.round(r.standard_normal((n, V)) * 8) / 4))
        self.tokens = r.integers(0, V, n)
        if V > 3:
            self.tokens[r.random(n) < 0.5] = 3           # the same token over again
        self.state = np.zeros((B, sk.splash_token_state_stride(V)), np.int64)
        hit = r.random((B, V)) < dense_state
        self.state[:, :V][hit] = r.integers(-32768, 32768, int(hit.sum()))
        self.rep, self.pres, self.freq = (r.choice(c, B) for c in
                                          ([1.0, 1.3, 0.8], [0.0, 0.5], [0.0, 0.25, -0.1]))
        self.bias = [[(int(r.integers(-2, V + 2)), float(r.standard_normal() * 3))
                      for _ in range(r.integers(0, nbias + 1))] for _ in range(B)]
        for b in self.bias:                               # an id listed twice
            if b:
                b.append((b[0][0], 2.5))
        words = (V + 31) // 32
        self.mask, self.rows = None, None
        if masks == "all":
            self.mask = r.integers(-2 ** 31, 2 ** 31, (n, words))
        elif masks == "some":
            self.mask = r.integers(-2 ** 31, 2 ** 31, (3, words))
            self.mask[1] = 0                              # leaves nothing
            self.rows = r.integers(-1, 3, n)

    def run(self, penal=True, bias=True, mask=True, out="new", max_block=None, **kw):
        n = self.n
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        logits = self.logits
        if out == "in place":
            logits = logits.clone(memory_format=torch.preserve_format) if logits.is_contiguous() \
                else logits._base.clone().as_strided(logits.size(), logits.stride(), logits.storage_offset())
            o = logits
        else:
            o = torch.full((n, self.V), 77.0, device="cuda") if out == "new" else None
        a = {}
        if penal:
            a = dict(block_tokens=i32(self.tokens), state=torch.tensor(self.state, device="cuda").short(),
                     repetition=f32(self.rep), presence=f32(self.pres), frequency=f32(self.freq))
        if bias:
            off = np.concatenate([[0], np.cumsum([len(b) for b in self.bias])])
            e = [x for b in self.bias for x in b]
            a |= dict(bias_offsets=i32(off), bias_ids=i32([x[0] for x in e]),
                      bias_values=f32([x[1] for x in e]))
        if mask and self.mask is not None:
            a |= dict(mask=torch.tensor(self.mask, device="cuda").int(),
                      mask_rows=None if self.rows is None else i32(self.rows))
        a |= kw
        ws = sk.alloc_target_workspace(n, self.V)
        sk.splash_choose_targets(logits, i32(self.q), got, ws, max_block or max(max(self.T), 1), out=o,
                                 device_status=st, **a)
        torch.cuda.synchronize()
        return got, o, st.item()

    def want(self, penal=True, bias=True, mask=True):
        return S.choose(self.logits.float().cpu().numpy(), self.q,
                        self.tokens if penal else None, self.state if penal else None, self.rep,
                        self.pres, self.freq, self.bias if bias else None,
                        self.mask if mask else None, self.rows)

    def check(self, **kw):
        out = kw.pop("out", "new")
        got, o, st = self.run(out=out, **kw)
        z, pick = self.want(**kw)
        live = np.zeros(self.n, bool)
        live[:self.q[-1]] = True
        g = got.cpu().numpy()
        assert np.array_equal(g[live], pick[live]), (g[live], pick[live])
        assert (g[~live] == -7).all() and st == 0
        if o is not None:
            oo = o.cpu().numpy()
            assert np.array_equal(oo[live], z[live], equal_nan=True)
            if out == "new":
                assert (oo[~live] == 77).all()


# vocabularies around a vector, a mask word, and the windows of 1024 to 4096
VOCABS = [1, 2, 7, 8, 31, 32, 33, 63, 64, 65, 1000, 1021, 1024, 1025, 2041, 2047, 2048, 2049, 4095,
          4096, 4099, 10001]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("V", VOCABS)
def test_everything_at_once(V, kind):
    s = Scene(V, [1, 0, 5, 2], V, kind, tail=2, masks="some")
    s.check()
    s.check(out=None)
    if kind == "f32":
        s.check(out="in place")


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("penal,bias,mask", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0)])
def test_each_step_alone(penal, bias, mask, kind):
    s = Scene(17, [3, 4], 2500, kind)
    s.check(penal=bool(penal), bias=bool(bias), mask=bool(mask))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("stride,start", [(2500, 1), (2501, 0), (2503, 3), (2560, 0), (2507, 5)])
def test_rows_at_any_alignment(stride, start, kind):
    s = Scene(stride + start, [2, 9], 2500, kind, stride=stride, start=start)
    s.check()
    if kind == "f32":
        s.check(out="in place")


@pytest.mark.parametrize("kind", list(KINDS))
def test_many_sequences_and_long_blocks(kind):
    s = Scene(3, [128, 1, 0, 127], 700, kind, masks="some", nbias=60)
    s.check()
    s = Scene(4, list(np.random.default_rng(1).integers(0, 4, 700)), 300, kind)
    s.check()


def test_windows_of_several_vectors():
    """Sequences times windows enough that a thread takes two or four vectors."""
    for kind, V, B in (("bf16", 40001, 80), ("bf16", 50003, 80), ("f16", 49152, 80),
                       ("f32", 20480, 80), ("f32", 16389, 60)):
        s = Scene(V, [1, 2] * (B // 2), V, kind, masks="some", dense_state=0.01, nbias=300)
        s.check(out="new")
        s.check(out=None)


def test_a_state_full_of_tokens():
    """Every token touched: the list of special tokens is the whole window."""
    for kind, V in (("bf16", 6000), ("f32", 3001), ("f32", 3000)):
        s = Scene(5, [2, 6], V, kind, dense_state=1.0)
        s.check()
        if kind == "f32":
            s.check(out="in place")


def test_single_penalties_and_values_that_do_not_count():
    s = Scene(6, [4, 4, 4], 900, "f32", masks="none")
    st = torch.tensor(s.state, device="cuda").short()
    for name, vals in (("repetition", [1.5, 0.0, float("nan")]), ("presence", [0.5, 0, 1]),
                       ("frequency", [0.1, 0, -2])):
        got, o, code = s.run(penal=False, bias=False, block_tokens=i32(s.tokens), state=st,
                             **{name: f32(vals)})
        z, pick = S.choose(s.logits.cpu().numpy(), s.q, s.tokens, s.state,
                           **{name: vals})
        assert np.array_equal(o.cpu().numpy(), z) and got.tolist() == list(pick) and code == 0


@pytest.mark.parametrize("kind", list(KINDS))
def test_infinities_nans_and_rows_without_a_choice(kind):
    s = Scene(7, [6], 3000, kind, masks="none", nbias=3)
    lo, inf, nan = torch.finfo(KINDS[kind]).min, float("inf"), float("nan")
    s.logits[0] = -inf
    s.logits[1] = nan
    s.logits[2, ::2] = nan
    s.logits[3] = lo
    s.logits[4, 100] = inf
    s.logits[5] = -inf
    s.logits[5, 2999] = lo
    s.check()
    s.check(penal=False, bias=False, mask=False)
    got, _, _ = s.run(penal=False, bias=False)
    assert got.tolist()[0] == -1 and got.tolist()[1] == -1 and got.tolist()[4] == 100
    # NaN and infinity where the mask closes
    s.mask = np.zeros((6, (3000 + 31) // 32), np.int64)
    s.mask[:, 5] = 1 << 3
    s.logits[:, 163] = torch.tensor([1, 2, 3, 4, 5, 6], dtype=KINDS[kind])
    s.check()
    assert s.run(penal=False, bias=False)[0].tolist() == [163] * 6


def test_signed_zeros_tie_at_the_lowest_index():
    z = torch.full((2, 300), -1.0, device="cuda")
    z[0, 7], z[0, 9] = -0.0, 0.0
    z[1, 290], z[1, 11] = 0.0, -0.0
    got = i32([5, 5])
    sk.splash_choose_targets(z, i32([0, 1, 2]), got, sk.alloc_target_workspace(2, 300), 1)
    assert got.tolist() == [7, 11]


def test_a_mask_row_that_is_not_there_allows_nothing():
    s = Scene(8, [3], 500, "f32", masks="some")
    s.rows = np.array([-1, 3, 0])
    got, o, st = s.run()
    z, pick = s.want()
    assert st == sk.DEVICE_BAD_LENGTH and got.tolist() == list(pick) and pick[1] == -1
    assert np.array_equal(o.cpu().numpy(), z)


def test_unusable_offsets_leave_their_rows():
    s = Scene(9, [2, 3, 2], 400, "bf16", masks="none")
    for q in ([0, 2, 5, 99], [0, 2, 1, 3], [-1, 2, 5, 7]):
        s.q = np.array(q)
        got, o, st = s.run(penal=False, bias=False, max_block=4)
        assert st == sk.DEVICE_BAD_LENGTH
        ok = [b for b in range(3) if 0 <= q[b] <= q[b + 1] <= 7 and q[b + 1] - q[b] <= 4]
        rows = [r for b in ok for r in range(q[b], q[b + 1])]
        want = s.logits.float().argmax(-1).tolist()
        assert all(got[r].item() == (want[r] if r in rows else -7) for r in range(7))
    s.q = np.array([0, 2, 5, 7])
    got, _, st = s.run(penal=False, bias=False, max_block=2)   # the middle block is too long
    assert st == sk.DEVICE_BAD_LENGTH and got.tolist()[2:5] == [-7] * 3 and -7 not in got.tolist()[:2]
    # bias offsets past the list: that sequence has no biases
    got, o, st = s.run(penal=False, bias=False, bias_offsets=i32([0, 1, 9, 9]),
                       bias_ids=i32([4, 5, 6]), bias_values=f32([90, 90, 90]))
    assert st == sk.DEVICE_BAD_LENGTH and got.tolist()[:2] == [4, 4] and 5 not in got.tolist()[2:]


def test_choices_are_the_same_every_time_and_after_another_call():
    s = Scene(10, [16] * 8, 9000, "bf16", masks="some", nbias=40)
    a, o, _ = s.run()
    Scene(11, [16] * 8, 9000, "bf16").run()
    for _ in range(3):
        b, p, _ = s.run()
        assert torch.equal(a, b) and torch.equal(o, p)


def test_a_captured_call_follows_its_inputs():
    s = Scene(12, [4, 4], 5000, "bf16", masks="none")
    tok, st = i32(s.tokens), torch.tensor(s.state, device="cuda").short()
    rep, q, ws = f32(s.rep), i32(s.q), sk.alloc_target_workspace(8, 5000)
    got = torch.zeros(8, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.splash_choose_targets(s.logits, q, got, ws, 4, block_tokens=tok, state=st, repetition=rep)
    for seed in (1, 2):
        s.logits.copy_(torch.tensor(np.random.default_rng(seed).standard_normal((8, 5000)) * 3))
        s.rep = np.array([1.2, 3.0]) * seed
        rep.copy_(f32(s.rep))
        g.replay()
        torch.cuda.synchronize()
        z, pick = S.choose(s.logits.float().cpu().numpy(), s.q, s.tokens, s.state, s.rep)
        assert got.tolist() == list(pick)


# ---------------------------------------------------------------------------
# history
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("lens,V", [([1], 1), ([0, 3, 70, 1], 65), ([5000, 1, 0, 900], 3001),
                                    ([2] * 1100, 90), ([40000], 50021), ([300] * 3, 200003)])
def test_history_matches_the_oracle(lens, V, prompt, reset):
    r = np.random.default_rng(V)
    n, B = sum(lens) + 3, len(lens)                       # three rows of no sequence
    q = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    tokens = (V * r.random(n) ** 4).astype(np.int64)
    tokens[r.random(n) < 0.01] = V
    tokens[r.random(n) < 0.01] = -1
    stride = sk.splash_token_state_stride(V)
    state = r.integers(-32768, 32768, (B, stride))
    state[:, ::3] = 32766
    for accepted in (None, r.integers(-1, 6, B)):
        d = torch.tensor(state, device="cuda").short()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sk.splash_token_state_add(i32(tokens), i32(q), d, V, prompt=prompt, reset=reset,
                                  accepted=None if accepted is None else i32(accepted),
                                  device_status=st)
        want = S.history(state, tokens, q, V, accepted, prompt, reset)
        assert np.array_equal(d.cpu().numpy(), want) and st.item() == 0


@pytest.mark.parametrize("reset", [False, True])
def test_counts_stop_at_their_largest(reset):
    tokens = i32([7] * 40000 + [8])
    d = sk.alloc_token_state(1, 64)
    d[0, 6], d[0, 8] = 5, -32768
    sk.splash_token_state_add(tokens, i32([0, 40001]), d, 64, reset=reset)
    assert d[0, 7].item() == 32767 and d[0, 6].item() == (0 if reset else 5)
    assert d[0, 8].item() == (1 if reset else 1 - 32768)


@pytest.mark.parametrize("reset", [False, True])
def test_history_of_unusable_offsets(reset):
    d = sk.alloc_token_state(3, 64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.splash_token_state_add(i32([1, 2, 3, 4]), i32([0, 2, 1, 4]), d, 64, reset=reset,
                              device_status=st)
    assert st.item() == sk.DEVICE_BAD_LENGTH and d[1].abs().sum().item() == 0
    assert d[0, 1].item() == 1


def test_a_workspace_that_is_too_small():
    z, q, got = torch.zeros((4, 5000), device="cuda"), i32([0, 4]), i32([-7] * 4)
    with pytest.raises(sk.SplashError) as e:
        sk.splash_choose_targets(z, q, got, torch.empty(64, dtype=torch.uint8, device="cuda"), 4)
    assert e.value.status == -3 and got.tolist() == [-7] * 4


def test_output_rows_of_any_stride():
    for kind, V, pad in (("bf16", 2500, 3), ("f32", 2499, 5), ("f32", 2500, 12)):
        s = Scene(13, [3, 2], V, kind, masks="some")
        wide = torch.full((s.n, V + pad), 77.0, device="cuda")
        got, _, st = s.run(out=None)
        t2 = torch.full((s.n,), -7, dtype=torch.int32, device="cuda")
        off = np.concatenate([[0], np.cumsum([len(b) for b in s.bias])])
        e = [x for b in s.bias for x in b]
        sk.splash_choose_targets(
            s.logits, i32(s.q), t2, sk.alloc_target_workspace(s.n, V), 3, block_tokens=i32(s.tokens),
            state=torch.tensor(s.state, device="cuda").short(), repetition=f32(s.rep),
            presence=f32(s.pres), frequency=f32(s.freq), bias_offsets=i32(off),
            bias_ids=i32([x[0] for x in e]), bias_values=f32([x[1] for x in e]),
            mask=torch.tensor(s.mask, device="cuda").int(), mask_rows=i32(s.rows), out=wide[:, :V])
        assert torch.equal(got, t2) and (wide[:, V:] == 77).all()
        assert np.array_equal(wide[:, :V].cpu().numpy(), s.want()[0])


def test_rows_before_the_first_sequence_and_a_long_bias_list():
    s = Scene(14, [2, 3], 900, "bf16", masks="none", nbias=0)
    s.bias = [[(v, 0.25 * (v % 7)) for v in range(-3, 903)] * 3, []]       # every token, thrice
    s.check()
    # offsets that begin past row 0 leave the rows before them
    q = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    sk.splash_choose_targets(s.logits, i32([2, 4, 5]), q, sk.alloc_target_workspace(5, 900), 2)
    assert q.tolist() == [-7, -7] + s.logits[2:].float().argmax(-1).tolist()


@pytest.mark.parametrize("kind,in_place", [("bf16", False), ("f32", False), ("f32", True)])
def test_rows_further_apart_than_32_bits(kind, in_place):
    """Row strides past 2^31 values: five rows begin up to 2^33 values apart."""
    T, V, far = [2, 3], 2500, 2 ** 31 + 8
    s = Scene(21, T, V, kind)
    wide = torch.empty(4 * far + V, dtype=KINDS[kind], device="cuda")
    rows = wide.as_strided((5, V), (far, 1))
    rows.copy_(s.logits)
    s.logits = rows
    z, pick = s.want()
    out = rows if in_place else torch.full((5, V), 77.0, device="cuda")
    off = np.concatenate([[0], np.cumsum([len(b) for b in s.bias])])
    e = [x for b in s.bias for x in b]
    got = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    sk.splash_choose_targets(rows, i32(s.q), got, sk.alloc_target_workspace(5, V), 3, i32(s.tokens),
                             torch.tensor(s.state, device="cuda").short(), f32(s.rep), f32(s.pres),
                             f32(s.freq), i32(off), i32([x[0] for x in e]), f32([x[1] for x in e]),
                             torch.tensor(s.mask, device="cuda").int(), out=out)
    assert np.array_equal(got.cpu().numpy(), pick)
    assert np.array_equal(out.cpu().numpy(), z)


@pytest.mark.parametrize("T,V", [([128] * 3, 5000), ([1] * 300, 1500), ([127, 1, 0, 64], 131072)])
def test_the_longest_blocks_and_many_sequences_of_one_row(T, V):
    Scene(22, T, V, "bf16", masks="some", tail=2).check()
