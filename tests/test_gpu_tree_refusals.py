"""What the binding of the tree operators refuses, each before anything runs."""
from __future__ import annotations

import os

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from speculative_verify_attention_kv_gb300 import build as _build  # noqa: E402

if not os.path.exists(_build.LIB):
    _build.build()

from speculative_verify_attention_kv_gb300 import splash_kv as sk  # noqa: E402

I, F, H = torch.int32, torch.float32, torch.bfloat16


def z(*shape, dtype=I):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def pool(layers=0, pages=4):
    return dict(zip(("k_pages", "v_pages", "k_scales", "v_scales"),
                    sk.alloc_pool(pages, 2, 128, num_layers=layers)))


CALLS = {
    "masks": (sk.splash_tree_masks, lambda: dict(
        parents=z(6) - 1, q_offsets=z(3), masks=z(6, 1), max_block_len=4, context_lens=z(2),
        depths=z(6), positions=z(6))),
    "attend": (sk.splash_verify_attention_tree, lambda: dict(
        q=z(6, 4, 128, dtype=H), page_table=z(2, 5), context_lens=z(2), block_lens=z(2),
        tree_masks=z(6, 1), sm_scale=0.1, max_block_len=4, out=z(6, 4, 128, dtype=H),
        lse=z(6, 4, dtype=F), workspace=sk.alloc_tree_workspace(2, 6, 4, 2, 128, 4), **pool())),
    "accept": (sk.splash_accept_tree, lambda: dict(
        block_tokens=z(6), parents=z(6) - 1, target_tokens=z(6), q_offsets=z(3), context_lens=z(2),
        accepted=z(2), next_tokens=z(2), path_rows=z(6), path_tokens=z(6), max_block_len=4,
        context_lens_out=z(2))),
    "compact": (sk.splash_kv_compact, lambda: dict(
        slots=z(6), path_rows=z(6), q_offsets=z(3), accepted=z(2), **pool())),
    "layers": (sk.splash_kv_compact, lambda: dict(
        slots=z(6), path_rows=z(6), q_offsets=z(3), accepted=z(2), **pool(3))),
    "logprobs": (sk.splash_token_logprobs, lambda: dict(
        logits=z(6, 100, dtype=H), workspace=sk.alloc_logprobs_workspace(6, 100), tokens=z(6),
        logprobs=z(6, dtype=F), entropy=z(6, dtype=F), top_ids=z(6, 4), top_logprobs=z(6, 4, dtype=F),
        rows=z(6))),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_the_call_itself_is_taken(name):
    f, args = CALLS[name]
    before = sk.splash_launch_count()
    f(**args())
    torch.cuda.synchronize()
    assert sk.splash_launch_count() > before


@pytest.mark.parametrize("name", list(CALLS))
def test_every_tensor_is_checked(name):
    """Each tensor in turn: of another type, on the host, not a tensor, a view with
    gaps, one entry too many."""
    f, args = CALLS[name]
    for key, t in args().items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = {"type": t.double(), "host": t.cpu(), "no tensor": 3}
        wide = torch.zeros((*t.shape, 2), dtype=t.dtype, device="cuda")[..., 0]
        if not wide.is_contiguous():
            wrong["gaps"] = wide
        if key not in ("workspace", "logits"):
            wrong["length"] = torch.zeros((t.shape[0] + 1, *t.shape[1:]), dtype=t.dtype, device="cuda")
        if key in ("k_pages", "v_pages"):
            wrong["length"] = pool(3 if name == "layers" else 0, 5)[key]
        if key in ("tree_masks", "masks"):
            wrong["words"] = z(6, 0)
        if t.dim() > 1:
            wrong["dims"] = t.flatten()
        if key == "logits":
            del wrong["gaps"]
            wrong["gaps inside rows"] = z(6, 200, dtype=H)[:, ::2]
        for what, bad in wrong.items():
            a = args()
            a[key] = bad
            before = sk.splash_launch_count()
            with pytest.raises((TypeError, ValueError, sk.SplashError)):
                f(**a)
            assert sk.splash_launch_count() == before, (key, what)


@pytest.mark.parametrize("name,drop", [
    ("masks", "context_lens"), ("logprobs", "tokens"), ("logprobs", "logprobs"),
    ("logprobs", "top_ids"), ("logprobs", "top_logprobs")])
def test_partners_that_are_missing(name, drop):
    f, args = CALLS[name]
    before = sk.splash_launch_count()
    with pytest.raises(ValueError):
        f(**dict(args(), **{drop: None}))
    assert sk.splash_launch_count() == before


@pytest.mark.parametrize("name,change", [
    ("masks", dict(max_block_len=257)), ("masks", dict(max_block_len=33)),
    ("attend", dict(max_block_len=257)), ("attend", dict(max_block_len=33)),
    ("attend", dict(sm_scale=0.0)), ("attend", dict(ctas=2000)), ("attend", dict(ctas=1000)),
    ("accept", dict(max_block_len=257)), ("accept", dict(max_block_len=-1))])
def test_values_that_are_refused(name, change):
    f, args = CALLS[name]
    before = sk.splash_launch_count()
    with pytest.raises(sk.SplashError):
        f(**dict(args(), **change))
    assert sk.splash_launch_count() == before


def test_pools_that_are_not_one_pool():
    f, args = CALLS["layers"]
    for key, t in (("v_pages", sk.alloc_pool(4, 2, 128, num_layers=3)[1]),
                   ("k_pages", pool()["k_pages"]), ("v_pages", pool()["v_pages"])):
        with pytest.raises((TypeError, ValueError)):
            f(**dict(args(), **{key: t}))
    a = args()
    a.update(k_pages=a["k_pages"][:0], v_pages=a["v_pages"][:0], k_scales=a["k_scales"][:0],
             v_scales=a["v_scales"][:0])
    with pytest.raises(ValueError):
        f(**a)
    # layers in the reverse order, or one layer several times
    a = args()
    a.update(k_pages=a["k_pages"][:1].expand(3, -1, -1, -1, -1),
             v_pages=a["v_pages"][:1].expand(3, -1, -1, -1, -1))
    with pytest.raises(sk.SplashError):
        f(**a)


def test_top_of_more_than_the_limit_and_a_small_workspace():
    f, args = CALLS["logprobs"]
    with pytest.raises(sk.SplashError):
        f(**dict(args(), top_ids=z(6, 33), top_logprobs=z(6, 33, dtype=F)))
    with pytest.raises(sk.SplashError):
        f(**dict(args(), workspace=args()["workspace"][:16].clone()))


def test_status_on_the_host_is_refused():
    for f, args in CALLS.values():
        with pytest.raises((TypeError, ValueError)):
            f(**args(), device_status=torch.zeros(1, dtype=I))
        with pytest.raises((TypeError, ValueError)):
            f(**args(), device_status=z(1, dtype=torch.int64))
