"""The operators of a verify step whose drafts form a tree, as measured cases.

In the order a step runs them: ancestor masks, depths and positions from the
nodes' parents (``masks``), attention of every node over its sequence's int8
paged cache and its own ancestors (``attend``), the accepted path through the
tree (``accept``), the accepted nodes' cache rows moved together in every layer
(``compact``), and the log probabilities of the emitted tokens with entropy and
the likeliest alternatives (``logprobs``).

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
        # One step of 16 requests with trees of 16 nodes: latency.
        dict(name="masks_step", op="masks", seqs=16, lo=16, hi=16, deep=False, mix=1),
        # A large batch of ragged trees, some of them nearly chains.
        dict(name="masks_batch", op="masks", seqs=500, lo=1, hi=120, deep=True, mix=2),
        # One chat request at a short context, small heads: latency.
        dict(name="tree_one", op="attend", seqs=1, ctx_lo=1900, ctx_hi=1900, lo=21, hi=21, hq=16,
             hkv=4, dim=64, deep=False, mix=3),
        # A ragged batch whose larger trees have more rows than one row block.
        dict(name="tree_ragged", op="attend", seqs=32, ctx_lo=256, ctx_hi=16384, lo=1, hi=64,
             hq=24, hkv=4, dim=256, deep=False, mix=4),
        # 16 agents at 32768 tokens each, trees of 16 nodes: the cache's bandwidth.
        dict(name="tree_16x32k", op="attend", seqs=16, ctx_lo=32768, ctx_hi=32768, lo=16, hi=16,
             hq=24, hkv=4, dim=256, deep=False, mix=5),
        # The accepted paths of one step of 16 requests: latency.
        dict(name="accept_step", op="accept", seqs=16, lo=16, hi=16, deep=False, mix=6),
        # And of a large ragged batch.
        dict(name="accept_batch", op="accept", seqs=500, lo=1, hi=120, deep=True, mix=7),
        # A four-layer draft model's cache after a step of 16 requests.
        dict(name="compact_draft", op="compact", seqs=16, lo=16, hi=16, layers=4, hkv=2, dim=128,
             mix=8),
        # The target's 48 layers after a step of a ragged batch.
        dict(name="compact_48", op="compact", seqs=64, lo=1, hi=64, layers=48, hkv=4, dim=256,
             mix=9),
        # One decoding request that asks for five alternatives: latency.
        dict(name="logprobs_one", op="logprobs", rows=1, vocab=32768, kind="bf16", top=5,
             masked=False, pick=False, mix=10),
        # The rows on accepted paths of 256, fp32 logits of an odd vocabulary under a grammar.
        dict(name="logprobs_path", op="logprobs", rows=256, vocab=100003, kind="fp32", top=20,
             masked=True, pick=True, mix=11),
        # Log probabilities of a 1500-token prompt.
        dict(name="logprobs_prompt", op="logprobs", rows=1500, vocab=131072, kind="bf16", top=20,
             masked=False, pick=False, mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["masks", "attend", "attend", "attend", "accept", "compact", "logprobs",
                     "logprobs"])
    mix = rng.randrange(1 << 30)
    if op in ("masks", "accept"):
        lo = rng.choice([1, 1, 8])
        return dict(op=op, seqs=_log_int(rng, 1, 500), lo=lo, hi=_log_int(rng, lo, 250),
                    deep=rng.random() < 0.5, mix=mix)
    if op == "attend":
        hkv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 6, 7, 8])
        dim = rng.choice([64, 128, 256])
        # the cache of the listed long case at most, rows within twice the ragged one's
        seqs = _log_int(rng, 1, 32)
        most = 16 * 32768 * 4 * 256 // (seqs * hkv * dim)
        ctx_hi = _log_int(rng, 64, max(64, min(65536, most) // 2))
        room = max(1, min(128, 32 * 64 * 6 * 4 * 16384 // (seqs * ctx_hi * hkv * group) // 2))
        hi = _log_int(rng, 1, room)
        return dict(op=op, seqs=seqs, ctx_lo=rng.choice([0, 1, 40, max(1, ctx_hi // 2)]),
                    ctx_hi=ctx_hi, lo=rng.choice([1, hi]), hi=hi, hq=hkv * group, hkv=hkv,
                    dim=dim, deep=rng.random() < 0.3, mix=mix)
    if op == "compact":
        hkv, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256])
        seqs, hi = _log_int(rng, 1, 128), _log_int(rng, 2, 128)
        most = 64 * 48 * 4 * 256 * 64 // (seqs * max(hi, 32) * hkv * dim)
        return dict(op=op, seqs=seqs, lo=1, hi=hi, layers=_log_int(rng, 1, max(1, min(80, most))),
                    hkv=hkv, dim=dim, mix=mix)
    vocab = _log_int(rng, 1000, 200000)
    return dict(op=op, rows=_log_int(rng, 1, max(1, 1500 * 131072 // vocab // 3)), vocab=vocab,
                kind=rng.choice(["bf16", "bf16", "fp16", "fp32"]), top=rng.choice([0, 1, 5, 20]),
                masked=rng.random() < 0.3, pick=rng.random() < 0.3, mix=mix)


def _lens(c):
    """Host lengths of a case: cached tokens and tree nodes of every request."""
    r = random.Random(c["mix"])
    ctx = [_log_int(r, max(1, c.get("ctx_lo", 100)), c.get("ctx_hi", 4000))
           for _ in range(c["seqs"])]
    T = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    if c.get("ctx_lo", 1) == 0:
        ctx[0] = 0                              # a request without a context yet
    return ctx, T


def _pages(n):
    return -(-n // PAGE)


def _words(c):
    return -(-c["hi"] // 32)


def work(c):
    if c["op"] == "logprobs":
        n, V = c["rows"], c["vocab"]
        m = -(-n // 2) if c["pick"] else n
        kept = m - m // 8 if c["pick"] else n
        e = 4 if c["kind"] == "fp32" else 2
        return dict(bytes=kept * (V * e + 4 + 8 + 8 * c["top"]) + 4 * m * c["pick"],
                    flops=kept * V * 5)
    ctx, T = _lens(c)
    n, B = sum(T), len(T)
    if c["op"] == "masks":
        return dict(bytes=n * (4 + 4 * _words(c) + 8) + 4 * (2 * B + 1), flops=0)
    if c["op"] == "accept":
        return dict(bytes=n * (12 + 8) + 4 * (B + 1) + 16 * B, flops=0)
    if c["op"] == "compact":
        moved = n // 5                          # a quarter of the nodes past the root
        row = c["layers"] * c["hkv"] * 2 * (c["dim"] + 4)
        return dict(bytes=2 * moved * row + 8 * n + 4 * (2 * B + 1), flops=0)
    d, keys = c["dim"], sum(x + t for x, t in zip(ctx, T))
    pairs = sum(t * (x + 1) for x, t in zip(ctx, T))
    return dict(bytes=keys * c["hkv"] * (2 * d + 8) + n * c["hq"] * (4 * d + 4)
                + 4 * n * _words(c) + 4 * sum(_pages(x + t) for x, t in zip(ctx, T)),
                flops=4 * d * c["hq"] * pairs)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(T):
    o = [0]
    for t in T:
        o.append(o[-1] + t)
    return o


def _of_rows(T):
    """Sequence and place in the tree of every packed row."""
    seq = torch.repeat_interleave(torch.arange(len(T), device=DEV), _i32(T).long())
    return seq, torch.arange(sum(T), device=DEV) - _i32(_offsets(T)[:-1]).long()[seq]


def _tree(c, T, g):
    """Parents of every node (within its tree, -1 at the root), before it in order."""
    _, t = _of_rows(T)
    u = torch.rand(len(t), generator=g, device=DEV)
    back = (t.clamp(max=4) if c["deep"] else t).float()
    parent = t - 1 - (u * back).long().clamp(max=255)
    return torch.where(t == 0, -1, parent.clamp(min=0)).int()


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)
    return {"masks": _prep_masks, "attend": _prep_attend, "accept": _prep_accept,
            "compact": _prep_compact, "logprobs": _prep_logprobs}[c["op"]](c, g)


def _prep_masks(c, g):
    ctx, T = _lens(c)
    n = sum(T)
    return dict(op="masks", parents=_tree(c, T, g), offsets=_i32(_offsets(T)), ctx=_i32(ctx),
                most=c["hi"], masks=torch.zeros((n, _words(c)), dtype=torch.int32, device=DEV),
                depths=torch.zeros(n, dtype=torch.int32, device=DEV),
                positions=torch.zeros(n, dtype=torch.int32, device=DEV))


def _tree_bits(parents, T, most):
    """[nodes, most] truth values: i is t or one of its ancestors (a tree at a time is dense)."""
    seq, t = _of_rows(T)
    up = torch.zeros((len(T), most, most), device=DEV)
    up[seq, t, t] = 1
    kids = parents >= 0
    up[seq[kids], t[kids], parents.long()[kids]] = 1
    for _ in range(max(1, (most - 1).bit_length())):        # paths of twice the length
        up = (torch.matmul(up, up) > 0).float()
    return up[seq, t] > 0


def _pack(bits):
    """Truth values [n, m] as int32 words of 32 bits."""
    n, m = bits.shape
    wide = torch.zeros((n, -(-m // 32) * 32), dtype=torch.int64, device=DEV)
    wide[:, :m] = bits
    word = (wide.view(n, -1, 32) << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(word >= 2 ** 31, word - 2 ** 32, word).int()


def _prep_attend(c, g):
    ctx, T = _lens(c)
    n, B, hkv, d = sum(T), len(T), c["hkv"], c["dim"]
    held = [_pages(x + t) for x, t in zip(ctx, T)]
    total, most = sum(held), max(held)
    pages = total + total // 16 + 3
    perm = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
    at = (_i32(_offsets(held)[:-1])[:, None] + torch.arange(most, device=DEV)).clamp(max=pages - 1)
    j = torch.arange(most, device=DEV)
    table = torch.where(j < _i32(held)[:, None], perm[at.long()], -1).int()
    # what a quantised normal row holds: codes of a third of the range, scales near 3 / 127
    codes = torch.empty((pages, hkv, 2, PAGE, d), dtype=torch.int8, device=DEV)
    codes.random_(-127, 128, generator=g)
    scales = 0.008 + 0.008 * torch.rand((2, pages, hkv, PAGE), generator=g, device=DEV)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = B * -(-c["hi"] * (c["hq"] // hkv) // 128)
    # scratch that a user's program keeps: two row blocks of partial sums an SM, and the plan
    scratch = 2 * 128 * sms * (d + 4) * 4 + 64 * (B + blocks + sms) + 65536
    return dict(op="attend", q=torch.randn((n, c["hq"], d), generator=g, device=DEV).bfloat16(),
                codes=codes, k_scales=scales[0].contiguous(), v_scales=scales[1].contiguous(),
                table=table.contiguous(), ctx=_i32(ctx), T=_i32(T), most=c["hi"],
                masks=_pack(_tree_bits(_tree(c, T, g), T, c["hi"])), sm_scale=d ** -0.5,
                out=torch.empty((n, c["hq"], d), dtype=torch.bfloat16, device=DEV),
                lse=torch.empty((n, c["hq"]), device=DEV),
                ws=torch.empty(scratch, dtype=torch.uint8, device=DEV))


def _prep_accept(c, g):
    ctx, T = _lens(c)
    n, B = sum(T), len(T)
    seq, t = _of_rows(T)
    parents = _tree(c, T, g)
    tokens = torch.randint(0, 50000, (n,), generator=g, device=DEV, dtype=torch.int32)
    # the target agrees with one of the children of most nodes
    first = torch.arange(n, device=DEV) - t
    liked = (torch.rand(n, generator=g, device=DEV) < 0.7) & (t > 0)
    child = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    above = (first + parents.long())[liked]
    child = child.scatter_reduce(0, above, torch.arange(n, device=DEV)[liked], "amax")
    other = torch.randint(0, 50000, (n,), generator=g, device=DEV, dtype=torch.int32)
    targets = torch.where(child >= 0, tokens[child.clamp(min=0)], other)
    new = lambda m: torch.empty(m, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(op="accept", tokens=tokens, parents=parents, targets=targets,
                offsets=_i32(_offsets(T)), ctx=_i32(ctx), most=c["hi"], ctx_out=new(B),
                accepted=new(B), following=new(B), path=new(n), path_tokens=new(n))


def _prep_compact(c, g):
    ctx, T = _lens(c)
    n, B, L = sum(T), len(T), c["layers"]
    seq, t = _of_rows(T)
    start = _i32([x % PAGE for x in ctx]).long()
    held = [_pages(x % PAGE + k) for x, k in zip(ctx, T)]
    pages = sum(held) + 2
    perm = torch.randperm(pages, generator=g, device=DEV)
    at = start[seq] + t
    slots = perm[_i32(_offsets(held)[:-1]).long()[seq] + at // PAGE] * PAGE + at % PAGE
    # a quarter of the nodes past the root is accepted, in order
    on = (torch.rand(n, generator=g, device=DEV) < 0.25) | (t == 0)
    count = torch.zeros(B, dtype=torch.int64, device=DEV).scatter_add(0, seq, on.long())
    rank = torch.cumsum(on.long(), 0) - 1
    first = torch.arange(n, device=DEV) - t
    path = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    path[(first + rank - rank[first])[on]] = torch.arange(n, device=DEV, dtype=torch.int32)[on]
    codes = torch.empty((L, pages, c["hkv"], 2, PAGE, c["dim"]), dtype=torch.int8, device=DEV)
    codes.random_(-127, 128, generator=g)
    scales = 0.008 + 0.008 * torch.rand((2, L, pages, c["hkv"], PAGE), generator=g, device=DEV)
    return dict(op="compact", codes=codes, k_scales=scales[0].contiguous(),
                v_scales=scales[1].contiguous(), slots=slots.int(), path=path,
                offsets=_i32(_offsets(T)), accepted=(count - 1).int())


def _prep_logprobs(c, g):
    n, V = c["rows"], c["vocab"]
    kind = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[c["kind"]]
    z = (3 * torch.randn((n, V), generator=g, device=DEV)).to(kind)
    tokens = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    if c["masked"]:
        # what a grammar shuts out; the emitted token is one that it allows
        z.masked_fill_(torch.rand((n, V), generator=g, device=DEV) < 0.8, -math.inf)
        z[torch.arange(n, device=DEV), tokens.long()] = 4
    rows, m = None, n
    if c["pick"]:
        # every other row is on an accepted path; -1 behind the end of a path
        i = torch.arange(0, n, 2, device=DEV, dtype=torch.int32)
        rows = torch.where(i // 2 % 8 == 7, -1, i)
        m = len(rows)
    f32 = torch.float32
    return dict(op="logprobs", z=z, tokens=tokens, rows=rows, top=c["top"],
                logprobs=torch.zeros(m, dtype=f32, device=DEV),
                entropy=torch.zeros(m, dtype=f32, device=DEV),
                top_ids=torch.zeros((m, c["top"]), dtype=torch.int32, device=DEV),
                top_logprobs=torch.zeros((m, c["top"]), dtype=f32, device=DEV),
                # scratch that a user's program keeps: 32 bytes a row and 512 tokens
                ws=torch.empty(32 * m * (V // 512 + 2), dtype=torch.uint8, device=DEV))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _own_masks(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_tree_masks(s["parents"], s["offsets"], s["masks"], s["most"], context_lens=s["ctx"],
                         depths=s["depths"], positions=s["positions"])
    return [s["masks"], s["depths"], s["positions"]]


def _own_attend(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_verify_attention_tree(s["q"], s["codes"][:, :, 0], s["codes"][:, :, 1],
                                    s["k_scales"], s["v_scales"], s["table"], s["ctx"], s["T"],
                                    s["masks"], s["sm_scale"], s["most"], s["out"], s["lse"],
                                    s["ws"])
    return [s["out"], s["lse"]]


def _own_accept(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_accept_tree(s["tokens"], s["parents"], s["targets"], s["offsets"], s["ctx"],
                          s["accepted"], s["following"], s["path"], s["path_tokens"], s["most"],
                          context_lens_out=s["ctx_out"])
    return [s["accepted"], s["following"], s["ctx_out"], s["path"], s["path_tokens"]]


def _own_compact(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_kv_compact(s["codes"][:, :, :, 0], s["codes"][:, :, :, 1], s["k_scales"],
                         s["v_scales"], s["slots"], s["path"], s["offsets"], s["accepted"])
    return [s["codes"], s["k_scales"], s["v_scales"]]


def _own_logprobs(s):
    from speculative_verify_attention_kv_gb300 import splash_kv as sk
    sk.splash_token_logprobs(s["z"], s["ws"], tokens=s["tokens"], logprobs=s["logprobs"],
                             entropy=s["entropy"], top_ids=s["top_ids"] if s["top"] else None,
                             top_logprobs=s["top_logprobs"] if s["top"] else None, rows=s["rows"])
    return [s["logprobs"], s["entropy"], s["top_ids"], s["top_logprobs"]]


_OWN = dict(masks=_own_masks, attend=_own_attend, accept=_own_accept, compact=_own_compact,
            logprobs=_own_logprobs)


def _places(offsets, n):
    """Sequence and place of every packed row, from the device's offsets."""
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(offsets.long(), row, right=True) - 1
    return seq, row - offsets.long()[seq]


def _closure(parents, seq, t, trees, most):
    """[nodes, most]: which places of its tree a node reaches going up, itself among them."""
    up = torch.zeros((trees, most, most), device=DEV)
    up[seq, t, t] = 1
    kid = (parents >= 0).float()
    up.index_put_((seq, t, parents.long().clamp(min=0)), kid, accumulate=True)
    for _ in range(max(1, (most - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    return up[seq, t] > 0


def _plain_masks(s):
    seq, t = _places(s["offsets"], len(s["parents"]))
    up = _closure(s["parents"], seq, t, len(s["ctx"]), s["most"])
    depth = up.sum(-1).int() - 1
    return [_pack(up), depth, s["ctx"][seq] + depth]


def _plain_attend(s):
    n, hq, d = s["q"].shape
    B, pages = s["table"].shape
    hkv, most = s["codes"].shape[1], s["most"]
    ctx, T = s["ctx"].long(), s["T"].long()
    at = s["table"].long().clamp(min=0)
    kv = s["codes"][at].permute(3, 0, 2, 1, 4, 5).reshape(2, B, hkv, pages * PAGE, d)
    k = kv[0].float() * s["k_scales"][at].transpose(1, 2).reshape(B, hkv, -1)[..., None]
    v = kv[1].float() * s["v_scales"][at].transpose(1, 2).reshape(B, hkv, -1)[..., None]
    offsets = torch.cumsum(T, 0) - T
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(offsets + T, row, right=True)
    t = row - offsets[seq]
    q = torch.zeros((B, most, hq, d), device=DEV)
    q[seq, t] = s["q"].float()
    q = q.view(B, most, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * s["sm_scale"]
    # context keys, and the tree's nodes by the rows' bits
    place = torch.arange(pages * PAGE, device=DEV) - ctx[:, None]
    node = place.clamp(0, most - 1)
    masks = torch.zeros((B, most, s["masks"].shape[1]), dtype=torch.int32, device=DEV)
    masks[seq, t] = s["masks"]
    words = masks.gather(2, (node // 32)[:, None].expand(B, most, -1))
    inside = ((place >= 0) & (place < T[:, None]))[:, None]
    seen = (place < 0)[:, None] | (inside & ((words >> (node % 32)[:, None]) & 1 > 0))
    seen = seen[:, None, :, None].expand(B, 1, most, hq // hkv, pages * PAGE).flatten(2, 3)
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = e.sum(-1, keepdim=True)
    v = torch.where((place < T[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.view(B, hkv, most, -1, d).transpose(1, 2).reshape(B, most, hq, d)
    lse = lse.view(B, hkv, most, -1).transpose(1, 2).reshape(B, most, hq)
    return [o[seq, t].to(torch.bfloat16), lse[seq, t]]


def _plain_accept(s):
    n, B = len(s["tokens"]), len(s["ctx"])
    seq, t = _places(s["offsets"], n)
    row = torch.arange(n, device=DEV)
    first = row - t
    above = (first + s["parents"].long()).clamp(min=0)
    fits = (s["parents"] >= 0) & (s["tokens"] == s["targets"][above])
    # of a node's fitting children the first one
    best = torch.full((n,), n, dtype=torch.int64, device=DEV)
    best = best.scatter_reduce(0, above, torch.where(fits, row, n), "amin")
    off = (t > 0) & (best[above] != row)
    dense = torch.zeros((B, s["most"]), dtype=torch.bool, device=DEV)
    dense[seq, t] = off
    # accepted: nothing on the way up is off it
    up = _closure(s["parents"], seq, t, B, s["most"])
    on = ~(up & dense[seq]).any(-1)
    rank = torch.cumsum(on.long(), 0) - 1
    count = torch.zeros(B, dtype=torch.int64, device=DEV).scatter_add(0, seq, on.long())
    to = torch.where(on, first + rank - rank[first], n)
    path = torch.full((n + 1,), -1, dtype=torch.int64, device=DEV).index_put((to,), row)[:n]
    path = torch.where(t < count[seq], path, -1)
    got = path.clamp(min=0)
    tokens = torch.where(path >= 0, s["tokens"][got], -1)
    last = path[s["offsets"][:-1].long() + count - 1]
    return [(count - 1).int(), s["targets"][last], (s["ctx"] + count).int(), path.int(), tokens]


def _plain_compact(s):
    n = len(s["slots"])
    seq, t = _places(s["offsets"], n)
    slots = s["slots"].long()
    moved = (t <= s["accepted"].long()[seq]) & (s["path"] >= 0)
    src = torch.where(moved, slots[s["path"].long().clamp(min=0)], slots)
    at = (slice(None), slots // PAGE, slice(None), slice(None), slots % PAGE)
    s["codes"][at] = s["codes"][:, src // PAGE, :, :, src % PAGE]
    for x in (s["k_scales"], s["v_scales"]):
        x[:, slots // PAGE, :, slots % PAGE] = x[:, src // PAGE, :, src % PAGE]
    return [s["codes"], s["k_scales"], s["v_scales"]]


def _plain_logprobs(s):
    keep = torch.ones_like(s["tokens"], dtype=torch.bool) if s["rows"] is None else s["rows"] >= 0
    at = torch.arange(len(s["z"]), device=DEV) if s["rows"] is None else s["rows"].long()
    at = at.clamp(min=0)
    z = s["z"].float() if s["rows"] is None else s["z"][at].float()
    V = z.shape[1]
    top = z.amax(-1, keepdim=True)
    t = z - top
    e = torch.exp(t)
    total = e.sum(-1)
    lse = torch.log(total)
    entropy = lse - (e * torch.where(e > 0, t, 0.0)).sum(-1) / total
    got = t.gather(1, s["tokens"][at].long()[:, None])[:, 0] - lse
    # the largest first, equal ones by index: both in one whole number
    bits = (z + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, -2147483648 - bits - 1, bits)
    key = bits * 2 ** 32 + (V - 1 - torch.arange(V, device=DEV))
    best = key.topk(s["top"], dim=1).values
    ids = V - 1 - (best & (2 ** 32 - 1))
    top_lp = t.gather(1, ids) - lse[:, None]
    ids = torch.where(top_lp > -math.inf, ids, -1).int()
    k2 = keep[:, None]
    return [torch.where(keep, got, s["logprobs"]), torch.where(keep, entropy, s["entropy"]),
            torch.where(k2, ids, s["top_ids"]), torch.where(k2, top_lp, s["top_logprobs"])]


_PLAIN = dict(masks=_plain_masks, attend=_plain_attend, accept=_plain_accept,
              compact=_plain_compact, logprobs=_plain_logprobs)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    if c["op"] in ("masks", "accept"):
        return None                     # whole numbers alone
    s = prepare(c, seed)
    return {"attend": _exact_attend, "compact": _exact_compact,
            "logprobs": _exact_logprobs}[c["op"]](s)


def _exact_attend(s):
    """Request by request, head by head: the keys that a node sees, and their weights."""
    hq, d = s["q"].shape[1:]
    hkv = s["codes"].shape[1]
    out, lse, row = torch.zeros_like(s["q"], dtype=torch.float64), s["lse"].double(), 0
    for b, (ctx, T) in enumerate(zip(s["ctx"].tolist(), s["T"].tolist())):
        pages = s["table"][b, :_pages(ctx + T)].long()
        bit = torch.arange(32 * s["masks"].shape[1], device=DEV)
        own_keys = (s["masks"][row:row + T].long()[:, bit // 32] >> (bit % 32)) & 1
        shut = torch.cat([torch.zeros((T, ctx), device=DEV, dtype=torch.bool),
                          own_keys[:, :T] == 0], 1)
        for h in range(hkv):
            kv = s["codes"][pages, h].double()              # [pages, 2, 16, d]
            k = (kv[:, 0] * s["k_scales"][pages, h].double()[..., None]).flatten(0, 1)[:ctx + T]
            v = (kv[:, 1] * s["v_scales"][pages, h].double()[..., None]).flatten(0, 1)[:ctx + T]
            heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
            x = torch.einsum("tgd,jd->tgj", s["q"][row:row + T, heads].double(), k)
            x = (x * s["sm_scale"]).masked_fill(shut[:, None], -math.inf)
            lse[row:row + T, heads] = torch.logsumexp(x, -1)
            out[row:row + T, heads] = torch.einsum("tgj,jd->tgd", torch.softmax(x, -1), v)
        row += T
    return [out, lse]


def _exact_compact(s):
    """Token by token of every path, in order; codes are whole numbers."""
    offsets, path, slots = s["offsets"].tolist(), s["path"].tolist(), s["slots"].tolist()
    src, dst = [], []
    for b, a in enumerate(s["accepted"].tolist()):
        for i in range(offsets[b], offsets[b] + a + 1):
            src.append(slots[path[i]])
            dst.append(slots[i])
    src, dst = torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV)
    both = []
    for x in (s["k_scales"], s["v_scales"]):
        flat = x.double().transpose(2, 3).flatten(1, 2)     # [layers, slots, heads]
        old = flat.clone()
        flat[:, dst] = old[:, src]
        both.append(flat.view(x.shape[0], x.shape[1], PAGE, -1).transpose(2, 3))
    return [None] + both


def _exact_logprobs(s):
    """Row by row, from the distribution itself."""
    k = s["top"]
    lp, ent = s["logprobs"].double(), s["entropy"].double()
    ids, tops = s["top_ids"].clone(), s["top_logprobs"].double()
    rows = range(len(lp)) if s["rows"] is None else s["rows"].tolist()
    for i, r in enumerate(rows):
        if r < 0:
            continue
        p = torch.log_softmax(s["z"][r].double(), 0)
        live = p[p > -math.inf]
        lp[i] = p[int(s["tokens"][r])]
        ent[i] = -(live.exp() * live).sum()
        if k:
            value, order = torch.sort(s["z"][r].double(), descending=True, stable=True)
            tops[i] = p[order[:k]]
            ids[i] = torch.where(value[:k] > -math.inf, order[:k], -1).int()
    return [lp, ent, ids, tops]
