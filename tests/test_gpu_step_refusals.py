"""What the binding of the step operators refuses, each before anything runs:
wrong types, layouts, shapes, devices, missing partners."""
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


def pool(pages=4, hkv=2, D=128):
    return dict(zip(("k_pages", "v_pages", "k_scales", "v_scales"), sk.alloc_pool(pages, hkv, D)))


CALLS = {
    "tables": (sk.splash_build_tables, lambda: dict(
        context_lens=z(3), block_lens=z(3), page_table=z(3, 5), page_counts=z(3), free_pages=z(7),
        free_count=z(1), q_offsets=z(4), new_offsets=z(4), positions=z(9), slots=z(9), num_pages=7)),
    "release": (sk.splash_release_pages, lambda: dict(
        keep_lens=z(3), page_table=z(3, 5), page_counts=z(3), free_pages=z(7), free_count=z(1),
        released_offsets=z(4))),
    "qkv": (sk.splash_qkv_append, lambda: dict(
        q=z(5, 4, 128, dtype=H), k=z(5, 2, 128, dtype=H), v=z(5, 2, 128, dtype=H),
        q_out=z(5, 4, 128, dtype=H), positions=z(5), slots=z(5) - 1, inv_freq=z(64, dtype=F),
        q_weight=z(128, dtype=F), k_weight=z(128, dtype=F), freq_axis=z(64), **pool())),
    "gather": (sk.splash_kv_gather, lambda: dict(
        slots=z(5), k_out=z(5, 2, 128, dtype=H), v_out=z(5, 2, 128, dtype=H), **pool())),
    "history": (sk.splash_token_state_add, lambda: dict(
        tokens=z(6), q_offsets=z(3), state=z(2, 128, dtype=torch.int16), vocab=100, accepted=z(2))),
    "choose": (sk.splash_choose_targets, lambda: dict(
        logits=z(6, 100, dtype=H), q_offsets=z(3), target_tokens=z(6),
        workspace=sk.alloc_target_workspace(6, 100), max_block_len=4, block_tokens=z(6),
        state=z(2, 128, dtype=torch.int16), repetition=z(2, dtype=F) + 1, presence=z(2, dtype=F),
        frequency=z(2, dtype=F), bias_offsets=z(3), bias_ids=z(4), bias_values=z(4, dtype=F),
        mask=z(6, 4), mask_rows=z(6), out=z(6, 100, dtype=F))),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_the_call_itself_is_taken(name):
    f, args = CALLS[name]
    f(**args())
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", list(CALLS))
def test_every_tensor_is_checked(name):
    """Each tensor in turn: of another type, on the host, not a tensor, a view
    with gaps, one entry too many."""
    f, args = CALLS[name]
    before = None
    for key, t in args().items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = {"type": t.double(), "host": t.cpu(), "no tensor": 3}
        wide = torch.zeros((*t.shape, 2), dtype=t.dtype, device="cuda")[..., 0]
        if not wide.is_contiguous():        # a view of one entry has no gaps
            wrong["gaps"] = wide
        if key not in ("free_pages", "workspace", "bias_ids", "tokens", "mask", "logits"):
            longer = torch.zeros((t.shape[0] + 1, *t.shape[1:]), dtype=t.dtype, device="cuda")
            wrong["length"] = longer
        if key in ("k_pages", "v_pages"):
            wrong["length"] = sk.alloc_pool(5, 2, 128)[0 if key == "k_pages" else 1]
        if key == "mask":
            wrong["words"] = z(6, 3)
        if key == "page_table":
            wrong["dims"] = z(15)
        for what, bad in wrong.items():
            a = args()
            a[key] = bad
            before = sk.splash_launch_count()
            with pytest.raises((TypeError, ValueError, sk.SplashError)):
                f(**a)
            assert sk.splash_launch_count() == before, (key, what)


@pytest.mark.parametrize("name,drop", [
    ("choose", ["state"]), ("choose", ["block_tokens"]), ("choose", ["bias_ids"]),
    ("choose", ["bias_values"]), ("choose", ["bias_offsets"]), ("choose", ["mask"]),
    ("qkv", ["positions"]),
])
def test_partners_that_are_missing(name, drop):
    f, args = CALLS[name]
    a = args()
    for k in drop:
        a[k] = None
    before = sk.splash_launch_count()
    with pytest.raises(ValueError):
        f(**a)
    assert sk.splash_launch_count() == before


@pytest.mark.parametrize("change", [
    dict(q=(5, 4, 128, 1)), dict(inv_freq=(72,)), dict(inv_freq=(4,)), dict(head=96)])
def test_qkv_shapes_that_are_not_supported(change):
    f, args = CALLS["qkv"]
    a = args()
    if "q" in change:                       # rows that begin off 16 bytes
        a["q"] = torch.zeros(5 * 4 * 128 + 1, dtype=H, device="cuda")[1:].view(5, 4, 128)
    elif "inv_freq" in change:
        a["inv_freq"] = z(*change["inv_freq"], dtype=F)
        a["freq_axis"] = None
    else:
        a = dict(a, q=z(5, 4, 96, dtype=H), k=z(5, 2, 96, dtype=H), v=z(5, 2, 96, dtype=H),
                 q_out=z(5, 4, 96, dtype=H), inv_freq=None, q_weight=None, k_weight=None,
                 **pool(D=96))
    with pytest.raises(sk.SplashError) as e:
        f(**a)
    assert e.value.status in (-1, -2)


def test_in_place_output_needs_fp32():
    _, args = CALLS["choose"]
    a = args()
    a["out"] = a["logits"]
    with pytest.raises(ValueError):
        sk.splash_choose_targets(**a)


def test_status_on_the_host_is_refused():
    for f, args in CALLS.values():
        with pytest.raises((TypeError, ValueError)):
            f(**args(), device_status=torch.zeros(1, dtype=I))
        with pytest.raises((TypeError, ValueError)):
            f(**args(), device_status=z(1, dtype=torch.int64))
