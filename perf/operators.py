"""The operators around a verify step, as measured cases.

Four groups, in the order a step runs them: page tables and slot maps from the
request lengths (``tables``, ``release``), the per-head norm, rotation and
quantised append of the projections (``qkv``), cached rows read back by slot
(``gather``), and the target's choices from penalised, masked logits with the
token history behind the penalties (``targets``, ``history``).

``own`` False computes each in its plain form with elementary torch
operations; True calls the library.
"""
import math
import random

import torch

own = False

PAGE = 16
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One scheduling step of a ragged batch: 64 requests with 512 to 131072
        # cached tokens, blocks of 1, 4, 8 or 16 verify tokens.
        dict(name="tables_step", op="tables", seqs=64, ctx_lo=512, ctx_hi=131072, block=0, mix=1),
        # Admission of 64 new requests: tables and slots of their whole prompts.
        dict(name="tables_admit", op="tables", seqs=64, ctx_lo=512, ctx_hi=131072, block=1, mix=2),
        # End of a batch: half the requests finished, the others trimmed to
        # what they have committed.
        dict(name="release_batch", op="release", seqs=64, ctx_lo=512, ctx_hi=131072, mix=3),
        # A four-token verify block of one request with fp32 projections,
        # paired (interleaved) rotation of half the head: latency.
        dict(name="qkv_block4", op="qkv", seqs=1, block=4, hq=8, hkv=2, dim=128, rot=64, axes=1,
             paired=True, fp32=True, norm=True, mix=4),
        # The verify step of the ragged batch, three position axes
        # (time, height, width).
        dict(name="qkv_ragged64", op="qkv", seqs=64, block=0, hq=24, hkv=4, dim=256, rot=256,
             axes=3, paired=False, fp32=False, norm=True, mix=5),
        # Prefill of a 32768-token prompt.
        dict(name="qkv_prompt32k", op="qkv", seqs=1, block=32768, hq=24, hkv=4, dim=256, rot=256,
             axes=1, paired=False, fp32=False, norm=True, mix=6),
        # The recent context of three requests to a fp32 check, odd lengths,
        # with a padded tail.
        dict(name="gather_small", op="gather", rows=2501, pad=27, hkv=2, dim=64, fp32=True, mix=7),
        # Four 32768-token contexts to a dense bf16 attention.
        dict(name="gather_4x32k", op="gather", rows=131072, pad=0, hkv=4, dim=256, fp32=False,
             mix=8),
        # One request, plain decode, penalties only: latency.
        dict(name="targets_one", op="targets", seqs=1, block=1, vocab=32768, kind="bf16",
             penal=True, bias=0, masks=0, out=False, mix=9),
        # 16 requests x 16 verify tokens, half of the rows under a grammar,
        # penalties and 300 biases each; the choices alone.
        dict(name="targets_16x16", op="targets", seqs=16, block=16, vocab=131072, kind="bf16",
             penal=True, bias=300, masks=2, out=False, mix=10),
        # The ragged batch with an odd vocabulary in fp32, processed logits
        # kept for a sampler.
        dict(name="targets_ragged_out", op="targets", seqs=64, block=0, vocab=100003, kind="fp32",
             penal=True, bias=20, masks=1, out=True, mix=11),
        # Token history of 16 requests resumed with up to 32768 tokens each.
        dict(name="history_resume", op="history", seqs=16, lo=512, hi=32768, vocab=131072,
             prompt=False, mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "release", "qkv", "qkv", "gather", "targets", "targets", "history"])
    mix = rng.randrange(1 << 30)
    if op in ("tables", "release"):
        c = dict(op=op, seqs=_log_int(rng, 1, 128), ctx_lo=rng.choice([1, 40, 512]),
                 ctx_hi=_log_int(rng, 600, 32768), mix=mix)
        if op == "tables":
            c["block"] = rng.choice([0, 0, 1])
        return c
    if op == "qkv":
        seqs = _log_int(rng, 1, 100)
        hkv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 6, 7, 8])
        dim = rng.choice([64, 128, 256])
        # head counts up to those of the listed prompt case
        while hkv * (group + 2) * dim > 32 * 256:
            group = max(1, group // 2)
            hkv = max(1, hkv // 2)
        block = rng.choice([0, 1, _log_int(rng, 1, max(1, 12000 // seqs))])
        return dict(op=op, seqs=seqs, block=block, hq=hkv * group, hkv=hkv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), axes=rng.choice([1, 1, 3]),
                    paired=rng.random() < 0.4, fp32=rng.random() < 0.3, norm=rng.random() < 0.8,
                    mix=mix)
    if op == "gather":
        return dict(op=op, rows=_log_int(rng, 1, 100000), pad=rng.choice([0, 0, 5, 300]),
                    hkv=rng.choice([1, 2, 3, 4]), dim=rng.choice([64, 128, 256]),
                    fp32=rng.random() < 0.3, mix=mix)
    if op == "targets":
        seqs = _log_int(rng, 1, 64)
        vocab = _log_int(rng, 1000, 131072)
        block = rng.choice([0, 1, rng.randint(2, 16)])
        return dict(op=op, seqs=seqs, block=block, vocab=vocab,
                    kind=rng.choice(["bf16", "bf16", "fp16", "fp32"]), penal=rng.random() < 0.7,
                    bias=rng.choice([0, 3, 300]), masks=rng.choice([0, 1, 2]),
                    out=rng.random() < 0.3 and seqs * (16 if block == 0 else block) <= 400,
                    mix=mix)
    return dict(op=op, seqs=_log_int(rng, 1, 32), lo=rng.choice([1, 100]),
                hi=_log_int(rng, 200, 32768), vocab=_log_int(rng, 1000, 131072),
                prompt=rng.random() < 0.5, mix=mix)


def _lens(c):
    """Host lengths of a case: (ctx, T) of the scheduling and verify cases."""
    r = random.Random(c["mix"])
    B = c["seqs"]
    ctx = [_log_int(r, c.get("ctx_lo", 1), c.get("ctx_hi", 4096)) for _ in range(B)]
    block = c.get("block", 0)
    T = [r.choice([1, 4, 8, 16]) if block == 0 else block for _ in range(B)]
    if c["op"] == "tables" and block == 1:      # admission: the whole prompt is new
        ctx, T = [0] * B, ctx
    return ctx, T


def _history_lens(c):
    r = random.Random(c["mix"])
    return [_log_int(r, c["lo"], c["hi"]) for _ in range(c["seqs"])]


def _pages(n):
    return -(-n // PAGE)


def work(c):
    if c["op"] == "tables":
        ctx, T = _lens(c)
        held = [_pages(x) for x in ctx]
        new = sum(max(0, _pages(x + t) - h) for x, t, h in zip(ctx, T, held))
        used = sum(_pages(x + t) - x // PAGE for x, t in zip(ctx, T))
        n, B = sum(T), len(T)
        return dict(bytes=4 * (3 * B + used + new) + 4 * (new + 2 * n + 3 * B + 3), flops=0)
    if c["op"] == "release":
        ctx, _ = _lens(c)
        n = sum(_pages(x) for x in ctx[::2])
        return dict(bytes=4 * (2 * n + 4 * len(ctx) + 2), flops=0)
    if c["op"] == "qkv":
        _, T = _lens(c)
        n, e = sum(T), 4 if c["fp32"] else 2
        d = c["dim"]
        read = n * (c["hq"] + 2 * c["hkv"]) * d * e + n * 4 * (1 + c["axes"])
        write = n * (c["hq"] * d * 2 + 2 * c["hkv"] * (d + 4)) + n * 2 * c["hkv"] * d * 2
        return dict(bytes=read + write, flops=n * (c["hq"] + 2 * c["hkv"]) * d * 8)
    if c["op"] == "gather":
        n, e = c["rows"], 4 if c["fp32"] else 2
        return dict(bytes=n * 2 * c["hkv"] * (c["dim"] * (1 + e) + 4) + 4 * (n + c["pad"]),
                    flops=n * 2 * c["hkv"] * c["dim"])
    if c["op"] == "targets":
        _, T = _lens(c)
        n, B, V = sum(T), len(T), c["vocab"]
        e = 4 if c["kind"] == "fp32" else 2
        b = n * V * e + 4 * n
        b += B * V * 2 + 12 * B if c["penal"] else 0
        b += B * c["bias"] * 8
        b += {0: 0, 1: n, 2: n // 2}[c["masks"]] * ((V + 31) // 32) * 4
        b += n * V * 4 if c["out"] else 0
        return dict(bytes=b, flops=n * V * 4)
    n, B = sum(_history_lens(c)), c["seqs"]
    return dict(bytes=4 * n + 2 * B * _stride(c["vocab"]) + 4 * B, flops=n)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _stride(vocab):
    """Entries of a token-history row: the vocabulary rounded up to 64."""
    return (vocab + 63) // 64 * 64


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(T):
    o = [0]
    for t in T:
        o.append(o[-1] + t)
    return o


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 11)
    return {"tables": _prep_tables, "release": _prep_tables, "qkv": _prep_qkv,
            "gather": _prep_gather, "targets": _prep_targets,
            "history": _prep_history}[c["op"]](c, g)


def _prep_tables(c, g):
    ctx, T = _lens(c)
    B = len(ctx)
    held = [_pages(x) for x in ctx]
    most = max(_pages(x + t) for x, t in zip(ctx, T)) + 1
    total = sum(held)
    pages = int((total + sum(_pages(x + t) for x, t in zip(ctx, T))) * 1.05) + 8
    perm = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
    off = _i32(_offsets(held)[:-1])
    j = torch.arange(most, device=DEV, dtype=torch.int32)
    counts = _i32(held)
    at = (off[:, None] + j).clamp_(max=pages - 1)
    table = torch.where(j < counts[:, None], perm[at.long()], torch.full_like(at, -1))
    free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    free[: pages - total] = perm[total:]
    s = dict(op=c["op"], ctx=_i32(ctx), T=_i32(T), table=table.contiguous(), counts=counts,
             free=free, free_count=_i32([pages - total]), pages=pages, n=sum(T),
             counts_out=torch.empty_like(counts), free_count_out=_i32([0]),
             offsets=torch.empty(B + 1, dtype=torch.int32, device=DEV),
             new=torch.empty(B + 1, dtype=torch.int32, device=DEV))
    if c["op"] == "tables":
        s["positions"] = torch.empty(s["n"], dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(s["n"], dtype=torch.int32, device=DEV)
    else:
        keep = [0 if b % 2 == 0 else max(0, x - 1) for b, x in enumerate(ctx)]
        s["keep"] = _i32(keep)
    return s


def _inv_freq(rot):
    return torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)],
                        dtype=torch.float64).float().to(DEV)


def _slots_of(ctx, T, perm):
    """Slots of every sequence's block, whole pages of ``perm`` one after another."""
    first, used = [], 0
    for x, t in zip(ctx, T):
        first.append(used)
        used += _pages(x % PAGE + t)
    seq = torch.repeat_interleave(torch.arange(len(T), device=DEV), _i32(T).long())
    t = torch.arange(sum(T), device=DEV) - _i32(_offsets(T)[:-1]).long()[seq]
    at = _i32(ctx).long()[seq] % PAGE + t
    slot = perm[_i32(first).long()[seq] + at // PAGE].long() * PAGE + at % PAGE
    return slot.int(), (_i32(ctx).long()[seq] + t).int()


def _prep_qkv(c, g):
    ctx, T = _lens(c)
    n, hq, hkv, d = sum(T), c["hq"], c["hkv"], c["dim"]
    used = sum(_pages(x % PAGE + t) for x, t in zip(ctx, T))
    pages = used + used // 8 + 4
    slots, pos = _slots_of(ctx, T, torch.randperm(pages, generator=g, device=DEV))
    kind = torch.float32 if c["fp32"] else torch.bfloat16
    # the projections come out of one product: q, k and v of a token side by side
    x = torch.randn((n, hq + 2 * hkv, d), generator=g, device=DEV).to(kind)
    x[:, :, 1] *= 8
    if c["axes"] > 1:
        # an image's tokens: the height and width axes run beside the time axis
        wide = 32
        pos = torch.stack([pos, pos // wide % wide, pos % wide]).contiguous()
    codes = torch.zeros((pages, hkv, 2, PAGE, d), dtype=torch.int8, device=DEV)
    half = c["rot"] // 2
    return dict(op="qkv", q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:], codes=codes,
                k_scales=torch.zeros((pages, hkv, PAGE), device=DEV),
                v_scales=torch.zeros((pages, hkv, PAGE), device=DEV), positions=pos, slots=slots,
                inv_freq=_inv_freq(c["rot"]),
                freq_axis=(torch.arange(half, device=DEV, dtype=torch.int32) % 3).contiguous()
                if c["axes"] > 1 else None,
                q_weight=(1 + 0.1 * torch.randn(d, generator=g, device=DEV)) if c["norm"] else None,
                k_weight=(1 + 0.1 * torch.randn(d, generator=g, device=DEV)) if c["norm"] else None,
                paired=c["paired"], eps=1e-6,
                q_out=torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV),
                k_out=torch.empty((n, hkv, d), dtype=torch.bfloat16, device=DEV),
                v_out=torch.empty((n, hkv, d), dtype=torch.bfloat16, device=DEV))


def _prep_gather(c, g):
    n, hkv, d = c["rows"], c["hkv"], c["dim"]
    pages = _pages(n) + 5
    perm = torch.randperm(pages, generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    slots = torch.full((n + c["pad"],), -1, dtype=torch.int32, device=DEV)
    slots[:n] = (perm[i // PAGE] * PAGE + i % PAGE).int()
    codes = torch.randint(-127, 128, (pages, hkv, 2, PAGE, d), generator=g, device=DEV,
                          dtype=torch.int8)
    scales = 0.01 + 0.02 * torch.rand((2, pages, hkv, PAGE), generator=g, device=DEV)
    kind = torch.float32 if c["fp32"] else torch.bfloat16
    out = torch.zeros((2, n + c["pad"], hkv, d), dtype=kind, device=DEV)
    return dict(op="gather", codes=codes, k_scales=scales[0].contiguous(),
                v_scales=scales[1].contiguous(), slots=slots, k_out=out[0], v_out=out[1])


def _prep_targets(c, g):
    ctx, T = _lens(c)
    B, n, V = len(T), sum(T), c["vocab"]
    kind = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[c["kind"]]
    rng = random.Random(c["mix"] + 1)
    s = dict(op="targets", logits=(4 * torch.randn((n, V), generator=g, device=DEV)).to(kind),
             offsets=_i32(_offsets(T)), most=max(T), vocab=V, state=None, repetition=None,
             presence=None, frequency=None, bias_offsets=None, bias_ids=None, bias_values=None,
             mask=None, mask_rows=None, out=None,
             tokens=torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32),
             targets=torch.empty(n, dtype=torch.int32, device=DEV), ws=None)
    if c["penal"]:
        # a few hundred committed tokens and a few thousand prompt tokens each
        st = torch.zeros((B, _stride(V)), dtype=torch.int32, device=DEV)
        hist = torch.randint(0, V, (B, 400), generator=g, device=DEV)
        st.scatter_add_(1, hist, torch.ones_like(hist, dtype=torch.int32))
        ask = torch.randint(0, V, (B, 2000), generator=g, device=DEV)
        seen = torch.zeros_like(st).scatter_(1, ask, 1)
        s["state"] = (st - 32768 * seen).to(torch.int16)
        s["repetition"] = torch.tensor([rng.choice([1.0, 1.1, 1.3]) for _ in range(B)], device=DEV)
        s["presence"] = torch.tensor([rng.choice([0.0, 0.5]) for _ in range(B)], device=DEV)
        s["frequency"] = torch.tensor([rng.choice([0.1, 0.25]) for _ in range(B)], device=DEV)
    if c["bias"]:
        k = min(c["bias"], V)
        ids = torch.rand((B, V), generator=g, device=DEV).topk(k, dim=1).indices
        s["bias_ids"] = ids.reshape(-1).int()
        s["bias_values"] = 4 * torch.randn(B * k, generator=g, device=DEV)
        s["bias_offsets"] = torch.arange(B + 1, device=DEV, dtype=torch.int32) * k
    if c["masks"]:
        # 1: a mask for every row; 2: masks for every other row, by index
        rows = n if c["masks"] == 1 else max(1, n // 2)
        words = (V + 31) // 32
        bits = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=g, device=DEV)
        also = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=g, device=DEV)
        s["mask"] = (bits & also).int()
        if c["masks"] == 2:
            r = torch.arange(n, device=DEV, dtype=torch.int32)
            s["mask_rows"] = torch.where((r % 2 == 1) & (r // 2 < rows), r // 2,
                                         torch.full_like(r, -1))
    if c["out"]:
        s["out"] = torch.empty((n, V), dtype=torch.float32, device=DEV)
    # scratch that a user's program keeps: 8 bytes a row and 1024 tokens
    s["ws"] = torch.empty(8 * n * (V // 1024 + 2), dtype=torch.uint8, device=DEV)
    return s


def _prep_history(c, g):
    lens = _history_lens(c)
    B, n, V = len(lens), sum(lens), c["vocab"]
    # a text's tokens: a few very frequent ones
    u = torch.rand(n, generator=g, device=DEV)
    tokens = (V * u ** 4).int().clamp_(max=V - 1)
    state = torch.randint(-32768, 32768, (B, _stride(V)), generator=g, device=DEV,
                          dtype=torch.int16)
    return dict(op="history", tokens=tokens, offsets=_i32(_offsets(lens)), state=state, vocab=V,
                prompt=c["prompt"])


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _own_tables(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_build_tables(s["ctx"], s["T"], s["table"], s["counts"], s["free"], s["free_count"],
                           s["offsets"], s["new"], s["positions"], s["slots"], s["pages"],
                           page_counts_out=s["counts_out"], free_count_out=s["free_count_out"])
    return [s["table"], s["counts_out"], s["free_count_out"], s["offsets"], s["new"],
            s["positions"], s["slots"]]


def _own_release(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_release_pages(s["keep"], s["table"], s["counts"], s["free"], s["free_count"],
                            s["new"], page_counts_out=s["counts_out"],
                            free_count_out=s["free_count_out"])
    return [s["free"], s["counts_out"], s["free_count_out"], s["new"]]


def _own_qkv(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    kp, vp = s["codes"][:, :, 0], s["codes"][:, :, 1]
    sk.splash_qkv_append(s["q"], s["k"], s["v"], s["q_out"], kp, vp, s["k_scales"], s["v_scales"],
                         s["positions"], s["slots"], inv_freq=s["inv_freq"],
                         q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                         freq_axis=s["freq_axis"], interleaved=s["paired"])
    sk.splash_kv_gather(kp, vp, s["k_scales"], s["v_scales"], s["slots"], s["k_out"], s["v_out"])
    return [s["q_out"], s["k_out"], s["v_out"]]


def _own_gather(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_kv_gather(s["codes"][:, :, 0], s["codes"][:, :, 1], s["k_scales"], s["v_scales"],
                        s["slots"], s["k_out"], s["v_out"])
    return [s["k_out"], s["v_out"]]


def _own_targets(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_choose_targets(s["logits"], s["offsets"], s["targets"], s["ws"], s["most"],
                             block_tokens=s["tokens"], state=s["state"],
                             repetition=s["repetition"], presence=s["presence"],
                             frequency=s["frequency"], bias_offsets=s["bias_offsets"],
                             bias_ids=s["bias_ids"], bias_values=s["bias_values"],
                             mask=s["mask"], mask_rows=s["mask_rows"], out=s["out"])
    return [s["targets"]] if s["out"] is None else [s["targets"], s["out"]]


def _own_history(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_token_state_add(s["tokens"], s["offsets"], s["state"], s["vocab"],
                              prompt=s["prompt"], reset=True)
    return [s["state"]]


_OWN = dict(tables=_own_tables, release=_own_release, qkv=_own_qkv, gather=_own_gather,
            targets=_own_targets, history=_own_history)


def _prefix(x):
    """Exclusive prefix sums, with the total at the end."""
    z = torch.zeros(1, dtype=torch.int64, device=x.device)
    return torch.cat([z, torch.cumsum(x, 0)])


def _plain_tables(s):
    ctx, T, held = s["ctx"].long(), s["T"].long(), s["counts"].long()
    offsets = _prefix(T)
    need = torch.where(T > 0, ((ctx + T + PAGE - 1) // PAGE - held).clamp(min=0), 0)
    incl = torch.cumsum(need, 0)
    given = torch.where(incl <= s["free_count"], need, 0)
    new = _prefix(given)
    counts = held + given
    j = torch.arange(s["table"].shape[1], device=DEV)
    take = s["free_count"] - 1 - (new[:-1, None] + j - held[:, None])
    fresh = (j >= held[:, None]) & (j < counts[:, None])
    table = torch.where(fresh, s["free"][take.clamp(0, s["pages"] - 1)], s["table"])
    row = torch.arange(s["n"], device=DEV)
    seq = torch.searchsorted(offsets, row, right=True) - 1
    pos = ctx[seq] + row - offsets[seq]
    ok = (ctx + T + PAGE - 1) // PAGE <= counts
    slot = torch.where(ok[seq], table[seq, pos // PAGE].long() * PAGE + pos % PAGE, -1)
    return [table, counts.int(), (s["free_count"] - new[-1]).int(), offsets.int(), new.int(),
            pos.int(), slot.int()]


def _plain_release(s):
    held = s["counts"].long()
    keep = torch.minimum(held, (s["keep"].long() + PAGE - 1) // PAGE)
    new = _prefix(held - keep)
    j = torch.arange(s["table"].shape[1], device=DEV)
    gone = (j >= keep[:, None]) & (j < held[:, None])
    # released entries to their places behind the list, the others to a spare one
    spare = s["pages"]
    to = torch.where(gone, s["free_count"] + new[:-1, None] + j - keep[:, None], spare)
    free = torch.cat([s["free"], s["free"][:1]])
    free = free.index_put((to.reshape(-1),), s["table"].reshape(-1))
    return [free[:spare], keep.int(), (s["free_count"] + new[-1]).int(), new.int()]


def _plain_rotated(x, w, cos, sin, s):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if s["paired"] else \
        (x[..., :half], x[..., half:2 * half])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if s["paired"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_codes(x):
    scale = x.abs().amax(-1, keepdim=True) / 127
    code = torch.round(x / torch.where(scale == 0, 1.0, scale)).clamp(-127, 127)
    return torch.where(scale == 0, 0.0, code).to(torch.int8), scale[..., 0]


def _plain_rows(s, half, scales):
    page, at = s["slots"].long().clamp(min=0) // PAGE, s["slots"].long().clamp(min=0) % PAGE
    return s["codes"][page, :, half, at].float() * s[scales][page, :, at][..., None]


def _plain_qkv(s):
    pos = s["positions"] if s["positions"].dim() == 2 else s["positions"][None]
    axis = s["freq_axis"].long() if s["freq_axis"] is not None else \
        torch.zeros(len(s["inv_freq"]), dtype=torch.int64, device=DEV)
    angle = pos[axis].double().T * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _plain_rotated(s["q"], s["q_weight"], cos, sin, s).to(torch.bfloat16)
    k = _plain_rotated(s["k"], s["k_weight"], cos, sin, s)
    page, at = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    kc, ks = _plain_codes(k)
    vc, vs = _plain_codes(s["v"].float())
    s["codes"][page, :, 0, at] = kc
    s["codes"][page, :, 1, at] = vc
    s["k_scales"][page, :, at] = ks
    s["v_scales"][page, :, at] = vs
    return [q, _plain_rows(s, 0, "k_scales").to(torch.bfloat16),
            _plain_rows(s, 1, "v_scales").to(torch.bfloat16)]


def _plain_gather(s):
    real = (s["slots"] >= 0)[:, None, None]
    k = torch.where(real, _plain_rows(s, 0, "k_scales").to(s["k_out"].dtype), s["k_out"])
    v = torch.where(real, _plain_rows(s, 1, "v_scales").to(s["v_out"].dtype), s["v_out"])
    return [k, v]


def _plain_targets(s):
    V, n = s["vocab"], s["logits"].shape[0]
    z = s["logits"].float()
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(s["offsets"], row, right=True) - 1
    if s["state"] is not None:
        st = s["state"][:, :V].int()
        count = (st & 32767)[seq]
        # the block's own tokens up to each row
        first = s["offsets"].long()[seq]
        t = torch.arange(s["most"], device=DEV)
        before = first[:, None] + t <= row[:, None]
        tok = s["tokens"].long()[torch.where(before, first[:, None] + t, 0)]
        count = count.scatter_add(1, tok, before.int())
        seen = (count > 0) | (st < 0)[seq]
        r = s["repetition"][seq][:, None]
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - s["frequency"][seq][:, None] * count
        z = z - s["presence"][seq][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        B = s["offsets"].shape[0] - 1
        e = torch.arange(s["bias_ids"].shape[0], device=DEV)
        of = torch.searchsorted(s["bias_offsets"], e, right=True) - 1
        dense = torch.zeros((B, V), device=DEV)
        dense = dense.index_put((of, s["bias_ids"].long()), s["bias_values"])
        z = z + dense[seq]
    if s["mask"] is not None:
        v = torch.arange(V, device=DEV)
        at = row if s["mask_rows"] is None else s["mask_rows"].long()
        bit = (s["mask"][at.clamp(min=0)][:, v // 32] >> (v % 32)) & 1
        z = torch.where((bit == 1) | (at < 0)[:, None], z, -math.inf)
    # the lowest index among the largest values; -1 where nothing is left
    top = z.amax(-1, keepdim=True)
    v = torch.arange(V, device=DEV, dtype=torch.int32)
    best = torch.where(z == top, v, V).amin(-1)
    targets = torch.where(top[:, 0] > -math.inf, best, -1).int()
    return [targets] if s["out"] is None else [targets, z]


def _plain_history(s):
    B, stride = s["state"].shape
    row = torch.arange(s["tokens"].shape[0], device=DEV)
    seq = torch.searchsorted(s["offsets"], row, right=True) - 1
    count = torch.zeros(B * stride, dtype=torch.int32, device=DEV)
    count = count.scatter_add(0, seq * stride + s["tokens"].long(), torch.ones_like(s["tokens"]))
    state = torch.where(count > 0, -32768, 0) if s["prompt"] else count.clamp(max=32767)
    return [state.view(B, stride).to(torch.int16)]


_PLAIN = dict(tables=_plain_tables, release=_plain_release, qkv=_plain_qkv, gather=_plain_gather,
              targets=_plain_targets, history=_plain_history)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    if c["op"] in ("tables", "release", "history"):
        return None                     # whole numbers alone
    s = prepare(c, seed)
    if c["op"] == "gather":
        return _exact_gather(s)
    if c["op"] == "qkv":
        return _exact_qkv(s)
    return _exact_targets(s) if s["out"] is not None else None


def _exact_gather(s):
    """Row i of the outputs holds code times scale of slot i; others stay."""
    flat = s["codes"].permute(2, 0, 3, 1, 4).flatten(1, 2)          # [2, slots, heads, dim]
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    both = []
    for half, name in ((0, "k_scales"), (1, "v_scales")):
        scale = s[name].transpose(1, 2).flatten(0, 1)[at].double()  # [rows, heads]
        out = s["k_out" if half == 0 else "v_out"].double()
        out[live] = flat[half][at].double() * scale.unsqueeze(-1)
        both.append(out)
    return both


def _exact_qkv(s):
    """Rotation as a product of complex numbers, the codes from 64-bit values."""
    n = s["slots"].shape[0]
    half = s["inv_freq"].shape[0]
    pos = s["positions"].reshape(-1, n).double()
    phase = torch.empty((n, half), dtype=torch.float64, device=DEV)
    for i in range(half):
        a = 0 if s["freq_axis"] is None else int(s["freq_axis"][i])
        phase[:, i] = pos[a] * s["inv_freq"][i].double()
    turn = torch.polar(torch.ones_like(phase), phase).unsqueeze(1)

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        x = x.clone()
        if s["paired"]:
            z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:-1], half, 2)
                                      .contiguous()) * turn
            x[..., :2 * half] = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * half)
        else:
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
            x[..., :half], x[..., half:2 * half] = z.real, z.imag
        return x

    def stored(x):
        step = x.abs().max(-1, keepdim=True).values / 127
        code = torch.where(step > 0, x / step, torch.zeros_like(x)).round().clamp(-127, 127)
        return code * step

    return [turned(s["q"], s["q_weight"]), stored(turned(s["k"], s["k_weight"])),
            stored(s["v"].double())]


def _exact_targets(s):
    """Sequence by sequence and row by row. The choice is made on values rounded
    to 32 bits after each step, as the operator defines it."""
    V = s["vocab"]
    offsets = s["offsets"].tolist()
    z64 = s["logits"].double()
    targets = torch.full((z64.shape[0],), -1, dtype=torch.int32, device=DEV)
    for b in range(len(offsets) - 1):
        if s["state"] is not None:
            st = s["state"][b, :V].long()
            prompt, count = st < 0, st % 32768
            r, p, f = (s[k][b].double() for k in ("repetition", "presence", "frequency"))
        for row in range(offsets[b], offsets[b + 1]):
            z = z64[row]
            w = z.clone()                       # rounded to 32 bits after each step
            if s["state"] is not None:
                count[int(s["tokens"][row])] += 1
                out, seen = count > 0, (count > 0) | prompt
                for x, narrow in ((z, False), (w, True)):
                    fit = (lambda y: y.float().double()) if narrow else (lambda y: y)
                    up, down = fit(x / r), fit(x * r)
                    y = torch.where(seen & (x > 0), up, torch.where(seen, down, x))
                    y = fit(y - fit(f * count))
                    x.copy_(fit(y - p * out))
            if s["bias_ids"] is not None:
                lo, hi = int(s["bias_offsets"][b]), int(s["bias_offsets"][b + 1])
                ids = s["bias_ids"][lo:hi].long()
                z[ids] += s["bias_values"][lo:hi].double()
                w[ids] = (w[ids] + s["bias_values"][lo:hi].double()).float().double()
            if s["mask"] is not None:
                m = row if s["mask_rows"] is None else int(s["mask_rows"][row])
                if m >= 0:
                    bits = (s["mask"][m].unsqueeze(1) >> torch.arange(32, device=DEV)) & 1
                    shut = bits.reshape(-1)[:V] == 0
                    z[shut] = -math.inf
                    w[shut] = -math.inf
            top = w.max()
            if top > -math.inf:
                targets[row] = int((w == top).nonzero()[0])
    return [targets, z64]
