"""Target choices of batches so large that a warp takes several segments of the
vocabulary in turn: state and biases of the next segment, the ring across segments,
the best choice carried over, short last runs.

The reference takes each step in 64 bits and rounds it to 32. The double rounding
changes nothing (53 >= 2 * 24 + 2 bits, quotients, products, sums and differences), so
logits and choices are compared for equality."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from oracle import step_oracle as S  # noqa: E402
from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SEGMENT = 1024
DEV = "cuda"


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Batch:
    def __init__(self, seed, T, V, kind, density, masks, nbias, low=0, penal=True):
        g = torch.Generator(device=DEV).manual_seed(seed)
        B, n = len(T), int(sum(T))
        self.T, self.V, self.B, self.n, self.penal = T, V, B, n, penal
        rand = lambda *s: torch.rand(s, generator=g, device=DEV)  # noqa: E731
        ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)  # noqa: E731
        # few distinct values: the largest one is in several segments
        self.logits = ((torch.randn((n, V), generator=g, device=DEV) * 8).round().clamp(-20, 20) / 4).to(KINDS[kind])
        self.q = i32(np.concatenate([[0], np.cumsum(T)]))
        self.seq = torch.repeat_interleave(torch.arange(B, device=DEV), i32(T).long())
        border = (torch.arange(V, device=DEV) + 9) % SEGMENT < 18
        hit = (rand(B, V) < density) | (border & (rand(B, V) < 0.5)) | (torch.arange(V, device=DEV) < low)
        self.state = torch.zeros((B, sk.splash_token_state_stride(V)), dtype=torch.int16, device=DEV)
        self.state[:, :V] = torch.where(hit, ints(-32768, 32768, B, V) % 40 - 20, 0).short()
        self.state[:, V:] = -1                       # nothing of it is the vocabulary's
        self.tokens = ints(0, V, n).int()
        self.tokens[rand(n) < 0.3] = SEGMENT         # on a border, over again
        pick = lambda *v: torch.tensor(v, device=DEV)[ints(0, len(v), B)]  # noqa: E731
        self.rep, self.pres, self.freq = pick(1.0, 1.3, 0.8), pick(0.0, 0.5), pick(0.0, 0.25, -0.1)
        self.bias_ids = torch.where(rand(B, nbias) < 0.2, ints(0, V // SEGMENT, B, nbias) * SEGMENT - 1,
                                    ints(-2, V + 2, B, nbias)).int() if nbias else None
        self.bias = torch.randn((B, max(nbias, 1)), generator=g, device=DEV) * 3
        words = (V + 31) // 32
        self.mask = self.rows = None
        if masks:
            m = n if masks == "all" else 7
            self.mask = ints(-2 ** 31, 2 ** 31, m, words).int()
            if masks == "some":
                self.mask[1] = 0
                self.rows = ints(-1, 7, n).int()

    def spans(self):
        """Several segments to a run, by the library's rule."""
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        units = min(sum(-(-max(self.T) // 8) for _ in self.T), self.B + self.n // 8)
        return units * (self.V // SEGMENT) // (64 * sms)

    def run(self, out):
        ws = sk.alloc_target_workspace(self.n, self.V)
        got = torch.full((self.n,), -7, dtype=torch.int32, device=DEV)
        z = self.logits.clone() if out == "in place" else self.logits
        o = z if out == "in place" else torch.full((self.n, self.V), 77.0, device=DEV) if out else None
        a = dict(block_tokens=self.tokens, state=self.state, repetition=self.rep, presence=self.pres,
                 frequency=self.freq) if self.penal else {}
        if self.bias_ids is not None:
            a |= dict(bias_offsets=i32(np.arange(self.B + 1) * self.bias_ids.shape[1]),
                      bias_ids=self.bias_ids.reshape(-1), bias_values=self.bias.reshape(-1))
        st = i32([0])
        sk.splash_choose_targets(z, self.q, got, ws, max(self.T), mask=self.mask, mask_rows=self.rows, out=o,
                                 device_status=st, **a)
        assert st.item() == 0
        return got, o

    def want(self):
        to32 = lambda x: x.float().double()  # noqa: E731
        V, n, seq = self.V, self.n, self.seq
        z = self.logits.double()
        if self.penal:
            st = self.state[:, :V].int()
            count, prompt = (st & 32767)[seq], (st < 0)[seq]
            for back in range(max(self.T)):          # the block's tokens up to the row
                row = torch.arange(n, device=DEV) - back
                ok = row >= self.q[:-1].long()[seq]
                count.scatter_add_(1, self.tokens[row.clamp(min=0)].long()[:, None], ok.int()[:, None])
            r, p, f = (t.double()[seq][:, None] for t in (self.rep, self.pres, self.freq))
            seen = (count > 0) | prompt
            y = torch.where(z > 0, to32(z / r), to32(z * r))
            z = torch.where(seen, y, z)
            z = to32(z - to32(f * count))
            z = torch.where(count > 0, to32(z - p), z)
        if self.bias_ids is not None:
            add = torch.zeros((self.B, V + 4), dtype=torch.float64, device=DEV)
            for e in range(self.bias_ids.shape[1]):  # the last entry of an id
                add.scatter_(1, self.bias_ids[:, e:e + 1].long() + 2, self.bias[:, e:e + 1].double())
            z = to32(z + add[seq][:, 2:V + 2])
        if self.mask is not None:
            v = torch.arange(V, device=DEV)
            at = torch.arange(n, device=DEV) if self.rows is None else self.rows.long()
            bit = (self.mask[at.clamp(min=0)][:, v // 32] >> (v % 32)) & 1
            z = torch.where((bit == 1) | (at < 0)[:, None], z, -torch.inf)
        top = z.amax(-1, keepdim=True)
        best = torch.where(z == top, torch.arange(V, device=DEV), V).amin(-1)
        return torch.where(top[:, 0] > -torch.inf, best, -1).int(), z.float()


def check(b, outs):
    pick, z = b.want()
    for out in outs:
        got, o = b.run(out)
        assert torch.equal(got, pick), (got != pick).nonzero()[:5]
        if o is not None:
            assert torch.equal(o, z)


def test_the_reference_itself():
    """Against the oracle, at a size that it can do."""
    b = Batch(1, [3, 1, 2], 2500, "f32", 0.1, "some", 40)
    bias = [[(int(v), float(x)) for v, x in zip(b.bias_ids[i], b.bias[i])] for i in range(3)]
    z, pick = S.choose(b.logits.cpu().numpy(), b.q.tolist(), b.tokens.tolist(), b.state.cpu().numpy(),
                       b.rep.cpu().numpy(), b.pres.cpu().numpy(), b.freq.cpu().numpy(), bias,
                       b.mask.cpu().numpy(), b.rows.tolist())
    got = b.want()
    assert got[0].tolist() == list(pick) and np.array_equal(got[1].cpu().numpy(), z)
    check(b, [None, "new", "in place"])


# runs of 2, 3, 4 and 5 segments, whole and with a shorter last one
CASES = [
    ([1] * 160, 131072), ([1] * 256, 131072), ([1] * 400, 100003), ([1] * 400, 131072), ([1] * 420, 131071),
    ([3, 1] * 110, 100003), ([8, 2, 0, 5] * 60, 131072), ([9, 1] * 90, 131080),
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("T,V", CASES, ids=lambda x: f"{len(x)}x{max(x)}" if isinstance(x, list) else str(x))
def test_several_segments_to_a_warp(T, V, kind):
    b = Batch(V + len(T), T, V, kind, 0.01, "some", 60)
    assert b.spans() >= 2
    check(b, [None, "new"] + (["in place"] if kind == "f32" else []))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("density,low", [(0.1, 0), (0.5, 0), (1.0, 0), (0.0, 3000)])
def test_dense_and_crowded_histories(density, low, kind):
    """More special tokens to a segment than a warp has lanes, twice over and all."""
    b = Batch(int(density * 10) + low, [1] * 180 + [3] * 4, 131071, kind, density, None, 20, low)
    assert b.spans() >= 2
    check(b, [None, "new"] + (["in place"] if kind == "f32" else []))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("penal,nbias,masks", [(False, 0, None), (False, 50, None), (False, 0, "all"), (True, 0, None)])
def test_each_step_alone(penal, nbias, masks, kind):
    b = Batch(5, [1] * 200, 101007, kind, 0.02, masks, nbias, penal=penal)
    assert b.spans() >= 2
    check(b, [None, "new"])


def test_ties_keep_the_lowest_index_across_segments_and_runs():
    for kind in KINDS:
        z = torch.full((320, 100003), -1.0, dtype=KINDS[kind], device=DEV)
        r = np.random.default_rng(7)
        want = []
        for row in range(320):
            at = np.sort(r.choice(100003, 4, replace=False))
            if row % 3 == 0:
                at[1] = min(at[0] // SEGMENT * SEGMENT + SEGMENT, 100002)      # the next segment's first
            z[row, torch.tensor(at, device=DEV)] = 2.5
            want.append(int(at.min()))
        got = i32([-7] * 320)
        sk.splash_choose_targets(z, i32(np.arange(321)), got, sk.alloc_target_workspace(320, 100003), 1)
        assert got.tolist() == want


def test_a_large_batch_is_the_same_every_time():
    b = Batch(9, [2] * 170, 131072, "bf16", 0.02, "some", 30)
    assert b.spans() >= 2
    first = b.run("new")
    for _ in range(3):
        again = b.run("new")
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
