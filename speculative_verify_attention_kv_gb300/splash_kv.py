"""Python binding of ``libsplashkv.so`` (ctypes; argument marshalling only).

The functions carry the C names. Tensors are torch CUDA tensors; the binding
checks dtype, device, shape and contiguity, passes raw device pointers and the
current CUDA stream, and raises :class:`SplashError` on a non-zero status. All
computation happens in the library's CUDA kernels: there is no fallback, and
importing this module fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsplashkv.so")

PAGE_SIZE = 16
DEVICE_BAD_PAGE = 1
DEVICE_BAD_LENGTH = 2
DEVICE_TIMEOUT = 3
DEVICE_OUT_OF_PAGES = 5
DEVICE_BAD_TREE = 6
PATH_AUTO, PATH_SIMT, PATH_TENSOR, PATH_TENSOR_T = 0, 1, 2, 3
# PATH_TENSOR: tensor-core kernel with the query rows on the MMA's M side (any
# head_dim of 128 / 256, up to 128 rows); PATH_TENSOR_T: the transposed kernel
# (keys on M, rows on N; head_dim 256, up to 96 rows per unit), which automatic
# mode picks whenever it applies


class SplashError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with speculative_verify_attention_kv_gb300.build.build()"
            " (there is no non-CUDA implementation)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.splash_status_string.restype = ctypes.c_char_p
    lib.splash_status_string.argtypes = [I]
    lib.splash_abi_version.restype = I
    lib.splash_tensor_path_supported.restype = I
    lib.splash_tensor_path_supported.argtypes = [I]
    lib.splash_launch_count.restype = ctypes.c_ulonglong
    lib.splash_launch_count.argtypes = []
    lib.splash_set_wait_limit_ns.restype = ctypes.c_ulonglong
    lib.splash_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.splash_kv_append.restype = I
    lib.splash_kv_append.argtypes = [P, P, I, P, P, P, P, P, I, P, P, I, I, I, I, I, P, P]
    lib.splash_kv_append_bf16.restype = I
    lib.splash_kv_append_bf16.argtypes = [P, P, I, P, P, P, P, P, I, P, P, I, I, I, I, I, P, P]
    lib.splash_accept_commit.restype = I
    lib.splash_accept_commit.argtypes = [P, P, I, P, P, P, P, I, P, P]
    lib.splash_verify_attention_workspace_size.restype = S
    lib.splash_verify_attention_workspace_size.argtypes = [I, I, I, I, I, I]
    attn = [P, I, P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, F, P, P, P, S, P, P]
    lib.splash_verify_attention.restype = I
    lib.splash_verify_attention.argtypes = attn
    lib.splash_verify_attention_tuned.restype = I
    lib.splash_verify_attention_tuned.argtypes = attn + [I, I]
    lib.splash_verify_attention_swa.restype = I
    lib.splash_verify_attention_swa.argtypes = attn[:18] + [I] + attn[18:] + [I, I]
    lib.splash_verify_attention_profiled.restype = I
    lib.splash_verify_attention_profiled.argtypes = attn + [I, I, P, P]
    lib.splash_verify_attention_shared_workspace_size.restype = S
    lib.splash_verify_attention_shared_workspace_size.argtypes = [I, I, I, I, I, I]
    # shared_lens follows block_lens
    attn_sh = attn[:10] + [P] + attn[10:]
    lib.splash_verify_attention_shared.restype = I
    lib.splash_verify_attention_shared.argtypes = attn_sh
    lib.splash_verify_attention_shared_profiled.restype = I
    lib.splash_verify_attention_shared_profiled.argtypes = attn_sh + [I, I, P, P]
    lib.splash_verify_attention_fixed_scratch_bytes.restype = S
    lib.splash_verify_attention_fixed_scratch_bytes.argtypes = []
    lib.splash_verify_attention_fixed_scratch.restype = I
    lib.splash_verify_attention_fixed_scratch.argtypes = attn[:20] + [P, P]
    L = ctypes.c_longlong
    lib.splash_build_tables.restype = I
    lib.splash_build_tables.argtypes = [P, P, I, I, I, I, P, I, P, P, P, I, P, P, P, P, P, P, P, P]
    lib.splash_build_tables_served.restype = I
    lib.splash_build_tables_served.argtypes = lib.splash_build_tables.argtypes[:18] + [P, P, P]
    lib.splash_release_pages.restype = I
    lib.splash_release_pages.argtypes = [P, I, P, I, I, P, P, P, I, P, P, P, P, P]
    lib.splash_qkv_append.restype = I
    lib.splash_qkv_append.argtypes = [P, P, P, I, I, L, L, L, L, L, L, I, I, I, P, P, F, P, P, I,
                                      I, F, P, I, P, P, P, P, P, P, I, I, P, P]
    lib.splash_kv_gather.restype = I
    lib.splash_kv_gather.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, I, P, P]
    lib.splash_token_state_stride.restype = I
    lib.splash_token_state_stride.argtypes = [I]
    lib.splash_token_state_add.restype = I
    lib.splash_token_state_add.argtypes = [P, I, P, I, P, P, L, I, I, I, P, P]
    lib.splash_choose_targets_workspace_size.restype = S
    lib.splash_choose_targets_workspace_size.argtypes = [I, I]
    lib.splash_choose_targets.restype = I
    lib.splash_choose_targets.argtypes = [P, I, L, I, I, P, I, I, P, P, L, P, P, P, P, P, P, I, P,
                                          L, I, P, P, L, P, P, S, P, P]
    lib.splash_tree_masks.restype = I
    lib.splash_tree_masks.argtypes = [P, I, P, P, I, I, P, I, P, P, P, P]
    lib.splash_verify_attention_tree_workspace_size.restype = S
    lib.splash_verify_attention_tree_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.splash_verify_attention_tree.restype = I
    lib.splash_verify_attention_tree.argtypes = attn[:10] + [P, I] + attn[10:] + [I]
    lib.splash_accept_tree.restype = I
    lib.splash_accept_tree.argtypes = [P, P, P, I, P, P, P, P, P, P, P, I, I, P, P]
    lib.splash_kv_compact.restype = I
    lib.splash_kv_compact.argtypes = [P, P, P, P, L, L, I, P, P, I, P, P, I, I, I, I, I, P, P]
    lib.splash_token_logprobs_workspace_size.restype = S
    lib.splash_token_logprobs_workspace_size.argtypes = [I, I]
    lib.splash_token_logprobs.restype = I
    lib.splash_token_logprobs.argtypes = [P, I, L, I, I, P, I, P, P, P, I, P, P, P, S, P, P]
    return lib


LIB = _load()
EXPORTED = ("splash_status_string", "splash_abi_version", "splash_tensor_path_supported",
            "splash_set_wait_limit_ns", "splash_launch_count",
            "splash_kv_append", "splash_kv_append_bf16", "splash_accept_commit",
            "splash_verify_attention_swa",
            "splash_verify_attention_workspace_size", "splash_verify_attention",
            "splash_verify_attention_tuned", "splash_verify_attention_profiled",
            "splash_verify_attention_shared_workspace_size", "splash_verify_attention_shared",
            "splash_verify_attention_shared_profiled",
            "splash_verify_attention_fixed_scratch_bytes", "splash_verify_attention_fixed_scratch",
            "splash_build_tables", "splash_build_tables_served", "splash_release_pages", "splash_qkv_append",
            "splash_kv_gather", "splash_token_state_stride", "splash_token_state_add",
            "splash_choose_targets_workspace_size", "splash_choose_targets", "splash_tree_masks",
            "splash_verify_attention_tree_workspace_size", "splash_verify_attention_tree",
            "splash_accept_tree", "splash_kv_compact", "splash_token_logprobs_workspace_size",
            "splash_token_logprobs")


def tensor_path_available(head_dim: int) -> bool:
    return bool(LIB.splash_tensor_path_supported(int(head_dim)))


def splash_launch_count() -> int:
    """Kernels the library has enqueued since it was loaded."""
    return int(LIB.splash_launch_count())


def splash_set_wait_limit_ns(ns: int) -> int:
    """Limit of each internal wait of the tensor-core kernel for later launches
    (0 = the default of 1 s); returns the previous limit."""
    return int(LIB.splash_set_wait_limit_ns(int(ns)))


def status_string(status: int) -> str:
    return LIB.splash_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: torch.Tensor, name: str, dtype, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {t.dim()}")


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def alloc_pool(num_pages: int, num_kv_heads: int, head_dim: int, device="cuda",
               num_layers: int = 0):
    """Zeroed paged pool in the library's layout: (k_pages, v_pages, k_scales,
    v_scales). The codes are one allocation [num_pages, Hkv, 2, P, D]; k_pages
    and v_pages are its [:, :, 0] and [:, :, 1] views ([num_pages, Hkv, P, D]
    each, K and V codes of a (page, KV head) adjacent). ``num_layers`` > 0: that
    many pools in one allocation, each tensor with a leading layer axis (the form
    that splash_kv_compact takes whole; index it for the calls of one layer)."""
    layers = (num_layers,) if num_layers > 0 else ()
    codes = torch.zeros((*layers, num_pages, num_kv_heads, 2, PAGE_SIZE, head_dim),
                        dtype=torch.int8, device=device)
    scales = (*layers, num_pages, num_kv_heads, PAGE_SIZE)
    return (codes[..., 0, :, :], codes[..., 1, :, :],
            torch.zeros(scales, dtype=torch.float32, device=device),
            torch.zeros(scales, dtype=torch.float32, device=device))


def _check_pool(k_pages, v_pages):
    """k_pages / v_pages: the two halves of one [num_pages, Hkv, 2, P, D] code pool."""
    for n, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int8 or not t.is_cuda or t.dim() != 4:
            raise TypeError(f"{n} must be a 4-D int8 CUDA tensor")
    num_pages, hkv, P, D = k_pages.shape
    want = (hkv * 2 * P * D, 2 * P * D, D, 1)
    if tuple(v_pages.shape) != tuple(k_pages.shape) or tuple(k_pages.stride()) != want \
            or tuple(v_pages.stride()) != want \
            or v_pages.data_ptr() != k_pages.data_ptr() + P * D:
        raise ValueError("k_pages / v_pages must be the [:, :, 0] / [:, :, 1] views of one "
                         "[num_pages, Hkv, 2, P, D] pool (see alloc_pool)")


def splash_kv_append(k_new, v_new, k_pages, v_pages, k_scales, v_scales, page_table,
                     context_lens, block_lens, device_status=None, stream=None) -> None:
    """k_new / v_new: float32 (splash_kv_append) or bfloat16 (splash_kv_append_bf16)."""
    if k_new.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("k_new must be float32 or bfloat16")
    _check(k_new, "k_new", k_new.dtype, 3)
    _check(v_new, "v_new", k_new.dtype, 3)
    _check_pool(k_pages, v_pages)
    for n, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _check(t, n, torch.float32, 3)
    _check(page_table, "page_table", torch.int32, 2)
    _check(context_lens, "context_lens", torch.int32, 1)
    _check(block_lens, "block_lens", torch.int32, 1)
    if device_status is not None:
        _check(device_status, "device_status", torch.int32)
    num_pages, hkv, P, D = k_pages.shape
    if tuple(v_pages.shape) != (num_pages, hkv, P, D) or tuple(k_new.shape[1:]) != (hkv, D) \
            or k_new.shape != v_new.shape:
        raise ValueError("shape mismatch between k_new/v_new and the pool")
    fn = LIB.splash_kv_append if k_new.dtype == torch.float32 else LIB.splash_kv_append_bf16
    st = fn(
        _ptr(k_new), _ptr(v_new), k_new.shape[0], _ptr(k_pages), _ptr(v_pages), _ptr(k_scales),
        _ptr(v_scales), _ptr(page_table), page_table.shape[1], _ptr(context_lens),
        _ptr(block_lens), context_lens.shape[0], hkv, D, P, num_pages, _ptr(device_status),
        _stream(stream))
    if st != 0:
        raise SplashError(st, "splash_kv_append")


def splash_accept_commit(block_tokens, target_tokens, block_lens, context_lens, accepted,
                         next_tokens, device_status=None, stream=None) -> None:
    """Advance context_lens (in place) by the accepted drafts plus one."""
    for n, t in (("block_tokens", block_tokens), ("target_tokens", target_tokens),
                 ("block_lens", block_lens), ("context_lens", context_lens),
                 ("accepted", accepted), ("next_tokens", next_tokens)):
        _check(t, n, torch.int32, 1)
    if device_status is not None:
        _check(device_status, "device_status", torch.int32)
    B = block_lens.shape[0]
    if context_lens.shape[0] != B or accepted.shape[0] != B or next_tokens.shape[0] != B \
            or target_tokens.shape != block_tokens.shape:
        raise ValueError("shape mismatch")
    st = LIB.splash_accept_commit(_ptr(block_tokens), _ptr(target_tokens), block_tokens.shape[0],
                                  _ptr(block_lens), _ptr(context_lens), _ptr(accepted),
                                  _ptr(next_tokens), B, _ptr(device_status), _stream(stream))
    if st != 0:
        raise SplashError(st, "splash_accept_commit")


def splash_verify_attention_workspace_size(num_seqs: int, num_q_tokens: int, num_q_heads: int,
                                           num_kv_heads: int, head_dim: int,
                                           max_block_len: int) -> int:
    return int(LIB.splash_verify_attention_workspace_size(
        num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, max_block_len))


def splash_verify_attention_shared_workspace_size(num_seqs: int, num_q_tokens: int,
                                                  num_q_heads: int, num_kv_heads: int,
                                                  head_dim: int, max_block_len: int) -> int:
    return int(LIB.splash_verify_attention_shared_workspace_size(
        num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, max_block_len))


def alloc_workspace(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, max_block_len,
                    device="cuda", ctas_per_class: int = 0, shared: bool = False) -> torch.Tensor:
    """Workspace for splash_verify_attention (``shared``: for the shared-prefix
    entry point)."""
    query = (splash_verify_attention_shared_workspace_size if shared
             else splash_verify_attention_workspace_size)
    n = query(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, max_block_len)
    if n == 0:
        raise ValueError("invalid shape for the workspace size query")
    if ctas_per_class > 0:   # a fixed CTA count may need more partial rows than the default
        rows = max_block_len * (num_q_heads // num_kv_heads)
        if shared:
            rows = max(rows, 128)
        n += 2 * rows * 2 * ctas_per_class * (head_dim + 1) * 4
    return torch.empty(n, dtype=torch.uint8, device=device)


def splash_verify_attention(q, k_pages, v_pages, k_scales, v_scales, page_table, context_lens,
                            block_lens, sm_scale: float, max_block_len: int, out, lse, workspace,
                            device_status=None, stream=None, path: int = PATH_AUTO,
                            ctas_per_class: int = 0, events=None, window: int = 0,
                            shared_lens=None) -> None:
    """``events``: optional (begin, end) torch.cuda.Event pair recorded around
    the attention kernels (the profiled entry point). ``window`` > 0: sliding
    window of that many keys (splash_verify_attention_swa). ``shared_lens``:
    int32 [num_seqs], keys each sequence shares with the one before it
    (splash_verify_attention_shared; the workspace from
    ``alloc_workspace(..., shared=True)``)."""
    _check(q, "q", torch.bfloat16, 3)
    _check(out, "out", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    _check_pool(k_pages, v_pages)
    for n, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _check(t, n, torch.float32, 3)
    _check(page_table, "page_table", torch.int32, 2)
    _check(context_lens, "context_lens", torch.int32, 1)
    _check(block_lens, "block_lens", torch.int32, 1)
    _check(workspace, "workspace", torch.uint8, 1)
    if device_status is not None:
        _check(device_status, "device_status", torch.int32)
    num_pages, hkv, P, D = k_pages.shape
    n_tok, hq, dq = q.shape
    if dq != D or tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (n_tok, hq):
        raise ValueError("shape mismatch between q, out, lse and the pool")
    args = (_ptr(q), n_tok, _ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales),
            _ptr(page_table), page_table.shape[1], _ptr(context_lens), _ptr(block_lens),
            context_lens.shape[0], hq, hkv, D, P, num_pages, int(max_block_len), float(sm_scale),
            _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(device_status),
            _stream(stream))
    if shared_lens is not None:
        _check(shared_lens, "shared_lens", torch.int32, 1)
        if shared_lens.shape[0] != context_lens.shape[0]:
            raise ValueError("shared_lens must have one entry per sequence")
        if window != 0:
            raise ValueError("shared_lens is taken only without a window")
        ev = [None, None] if events is None else [
            ctypes.c_void_p(e.cuda_event) if e is not None else None for e in events]
        st = LIB.splash_verify_attention_shared_profiled(*args[:10], _ptr(shared_lens), *args[10:],
                                                         int(path), int(ctas_per_class), *ev)
    elif window != 0:
        if events is not None:
            raise ValueError("events are recorded only without a window")
        st = LIB.splash_verify_attention_swa(*args[:18], int(window), *args[18:], int(path),
                                             int(ctas_per_class))
    elif events is not None:
        ev = [ctypes.c_void_p(e.cuda_event) if e is not None else None for e in events]
        st = LIB.splash_verify_attention_profiled(*args, int(path), int(ctas_per_class), *ev)
    elif path == PATH_AUTO and ctas_per_class == 0:
        st = LIB.splash_verify_attention(*args)
    else:
        st = LIB.splash_verify_attention_tuned(*args, int(path), int(ctas_per_class))
    if st != 0:
        raise SplashError(st, "splash_verify_attention")


def splash_verify_attention_fixed_scratch(q, k_pages, v_pages, k_scales, v_scales, page_table,
                                          context_lens, block_lens, sm_scale: float,
                                          max_block_len: int, out, lse, device_status=None,
                                          stream=None) -> None:
    """splash_verify_attention with the library's fixed device scratch instead
    of a workspace (for callers that cannot allocate device memory)."""
    _check(q, "q", torch.bfloat16, 3)
    _check(out, "out", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    _check_pool(k_pages, v_pages)
    for n, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _check(t, n, torch.float32, 3)
    _check(page_table, "page_table", torch.int32, 2)
    _check(context_lens, "context_lens", torch.int32, 1)
    _check(block_lens, "block_lens", torch.int32, 1)
    if device_status is not None:
        _check(device_status, "device_status", torch.int32)
    num_pages, hkv, P, D = k_pages.shape
    n_tok, hq, dq = q.shape
    if dq != D or tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (n_tok, hq):
        raise ValueError("shape mismatch between q, out, lse and the pool")
    st = LIB.splash_verify_attention_fixed_scratch(
        _ptr(q), n_tok, _ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales),
        _ptr(page_table), page_table.shape[1], _ptr(context_lens), _ptr(block_lens),
        context_lens.shape[0], hq, hkv, D, P, num_pages, int(max_block_len), float(sm_scale),
        _ptr(out), _ptr(lse), _ptr(device_status), _stream(stream))
    if st != 0:
        raise SplashError(st, "splash_verify_attention_fixed_scratch")


# ---------------------------------------------------------------------------
# The rest of a verify step: page tables, projections into the cache, target
# choices. A step calls each of these once per layer or once per step, so the
# checks are one pass over a tensor list; _check words the errors.
# ---------------------------------------------------------------------------
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _check_all(specs, device_status) -> int:
    """specs: (tensor or None, name, dtype, ndim) of contiguous CUDA tensors, all
    on the current device. Returns the device index."""
    dev = torch.cuda.current_device()
    try:
        for t, name, dtype, ndim in specs:
            if t is not None and (t.dtype is not dtype or t.get_device() != dev
                                  or t.dim() != ndim or not t.is_contiguous()):
                break
        else:
            if device_status is None:
                return dev
    except AttributeError:
        pass
    for t, name, dtype, ndim in specs:           # the same with words
        if t is not None:
            _check(t, name, dtype, ndim)
            if t.get_device() != dev:
                raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if device_status is not None:
        _check(device_status, "device_status", torch.int32)
        if device_status.get_device() != dev or device_status.numel() < 1:
            raise ValueError("device_status must be an int32 tensor on the current device")
    return dev


def _tensors(**named) -> None:
    for name, t in named.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def _raw_stream(stream, dev: int) -> int:
    # the raw handle: a Stream object for the current stream costs 2.8 us of
    # host time a call, a fifth of a small call's whole
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _data(t):
    return None if t is None else t.data_ptr()


def _pool_on(k_pages, v_pages, dev: int):
    """Shape (num_pages, Hkv, P, D) of a pool on device ``dev``."""
    try:
        n, hkv, P, D = shape = k_pages.shape
        if k_pages.dtype is torch.int8 and v_pages.dtype is torch.int8 and v_pages.shape == shape \
                and k_pages.stride() == v_pages.stride() == (hkv * 2 * P * D, 2 * P * D, D, 1) \
                and v_pages.data_ptr() == k_pages.data_ptr() + P * D \
                and k_pages.get_device() == dev:
            return shape
    except ValueError:                           # not four dimensions
        pass
    _check_pool(k_pages, v_pages)
    raise ValueError(f"the pool is not on the current device, cuda:{dev}")


def splash_build_tables(context_lens, block_lens, page_table, page_counts, free_pages, free_count,
                        q_offsets, new_offsets, positions, slots, num_pages: int,
                        page_counts_out=None, free_count_out=None, device_status=None,
                        stream=None, served_lens=None) -> None:
    """Pages for the block of every sequence, positions and slots of its tokens.
    ``page_counts`` and ``free_count`` are updated in place unless their
    ``_out`` tensors are given. ``positions`` / ``slots``: int32 [num_tokens],
    possibly longer than sum(block_lens) (the tail gets slot -1). With
    ``served_lens`` (int32 [num_seqs], may be ``block_lens``) the block lengths of
    the sequences that got their pages, 0 of the others, and rows packed by them:
    what the rest of the step takes in place of ``block_lens``."""
    counts_out = page_counts if page_counts_out is None else page_counts_out
    free_out = free_count if free_count_out is None else free_count_out
    i32 = torch.int32
    dev = _check_all(((context_lens, "context_lens", i32, 1), (block_lens, "block_lens", i32, 1),
                      (page_table, "page_table", i32, 2), (page_counts, "page_counts", i32, 1),
                      (counts_out, "page_counts_out", i32, 1), (free_pages, "free_pages", i32, 1),
                      (free_count, "free_count", i32, 1), (free_out, "free_count_out", i32, 1),
                      (q_offsets, "q_offsets", i32, 1), (new_offsets, "new_offsets", i32, 1),
                      (positions, "positions", i32, 1), (slots, "slots", i32, 1),
                      (served_lens, "served_lens", i32, 1)), device_status)
    B, n = context_lens.shape[0], slots.shape[0]
    if block_lens.shape[0] != B or page_table.shape[0] != B or page_counts.shape[0] != B \
            or counts_out.shape[0] != B or q_offsets.shape[0] != B + 1 \
            or new_offsets.shape[0] != B + 1 or positions.shape[0] != n \
            or free_count.shape[0] != 1 or free_out.shape[0] != 1 \
            or (served_lens is not None and served_lens.shape[0] != B):
        raise ValueError("shape mismatch between the lengths, tables, offsets and slots")
    args = (
        context_lens.data_ptr(), block_lens.data_ptr(), B, n, PAGE_SIZE, int(num_pages),
        page_table.data_ptr(), page_table.shape[1], page_counts.data_ptr(), counts_out.data_ptr(),
        free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), free_out.data_ptr(),
        q_offsets.data_ptr(), new_offsets.data_ptr(), positions.data_ptr(), slots.data_ptr())
    end = _data(device_status), _raw_stream(stream, dev)
    if served_lens is None:
        st = LIB.splash_build_tables(*args, *end)
    else:
        st = LIB.splash_build_tables_served(*args, served_lens.data_ptr(), *end)
    if st != 0:
        raise SplashError(st, "splash_build_tables")


def splash_release_pages(keep_lens, page_table, page_counts, free_pages, free_count,
                         released_offsets, page_counts_out=None, free_count_out=None,
                         device_status=None, stream=None) -> None:
    """The pages past ``keep_lens`` tokens of every sequence back on the free
    list (its length is its capacity)."""
    counts_out = page_counts if page_counts_out is None else page_counts_out
    free_out = free_count if free_count_out is None else free_count_out
    i32 = torch.int32
    dev = _check_all(((keep_lens, "keep_lens", i32, 1), (page_table, "page_table", i32, 2),
                      (page_counts, "page_counts", i32, 1), (counts_out, "page_counts_out", i32, 1),
                      (free_pages, "free_pages", i32, 1), (free_count, "free_count", i32, 1),
                      (free_out, "free_count_out", i32, 1),
                      (released_offsets, "released_offsets", i32, 1)), device_status)
    B = keep_lens.shape[0]
    if page_table.shape[0] != B or page_counts.shape[0] != B or counts_out.shape[0] != B \
            or released_offsets.shape[0] != B + 1 or free_count.shape[0] != 1 \
            or free_out.shape[0] != 1:
        raise ValueError("shape mismatch between the lengths, tables and offsets")
    st = LIB.splash_release_pages(
        keep_lens.data_ptr(), B, page_table.data_ptr(), page_table.shape[1], PAGE_SIZE,
        page_counts.data_ptr(), counts_out.data_ptr(), free_pages.data_ptr(),
        free_pages.shape[0], free_count.data_ptr(), free_out.data_ptr(),
        released_offsets.data_ptr(), _data(device_status), _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_release_pages")


def splash_qkv_append(q, k, v, q_out, k_pages, v_pages, k_scales, v_scales, positions, slots,
                      inv_freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                      freq_axis=None, interleaved: bool = False, rope_scale: float = 1.0,
                      device_status=None, stream=None) -> None:
    """Norm (with a weight), rotation (with ``inv_freq``, R/2 values) and
    quantised append. ``q``, ``k``, ``v``: float32 or bfloat16 [n, heads, D],
    strided views with contiguous rows. ``positions``: int32 [n] or [axes, n]
    (None without a rotation)."""
    _tensors(q=q, k=k, v=v, k_pages=k_pages, v_pages=v_pages)
    f32, i32 = torch.float32, torch.int32
    dev = _check_all(((q_out, "q_out", torch.bfloat16, 3), (k_scales, "k_scales", f32, 3),
                      (v_scales, "v_scales", f32, 3), (slots, "slots", i32, 1),
                      (inv_freq, "inv_freq", f32, 1), (q_weight, "q_weight", f32, 1),
                      (k_weight, "k_weight", f32, 1), (freq_axis, "freq_axis", i32, 1)),
                     device_status)
    pool = num_pages, hkv, P, D = _pool_on(k_pages, v_pages, dev)
    dt = q.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError("q must be float32 or bfloat16")
    strides = []
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dtype is not dt or t.dim() != 3 or t.get_device() != dev:
            raise TypeError(f"{name} must be a 3-D {dt} tensor on cuda:{dev}")
        st = t.stride()
        if st[2] != 1:
            raise ValueError(f"the rows of {name} must be contiguous")
        # along an axis of one the stride says nothing
        strides += [st[0] if t.shape[0] > 1 else 0, st[1] if t.shape[1] > 1 else 0]
    n, hq, _ = q.shape
    if q_out.shape != (n, hq, D) or q_out.shape != q.shape or k.shape != (n, hkv, D) \
            or v.shape != k.shape or slots.shape[0] != n or k_scales.shape != pool[:3] \
            or v_scales.shape != pool[:3]:
        raise ValueError("shape mismatch between q, k, v, q_out, slots and the pool")
    for w in (q_weight, k_weight):
        if w is not None and w.shape[0] != D:
            raise ValueError("a norm weight has one value per head dimension")
    half, axes = 0, 1
    if inv_freq is not None:
        half = inv_freq.shape[0]
        if positions is None:
            raise ValueError("a rotation needs positions")
        if not isinstance(positions, torch.Tensor) or positions.dtype is not i32 or positions.get_device() != dev \
                or not positions.is_contiguous():
            _check_all(((positions, "positions", i32, None),), None)
        if positions.dim() == 2:
            axes = positions.shape[0]
        if positions.dim() not in (1, 2) or positions.shape[-1] != n or axes < 1 \
                or (freq_axis is not None and freq_axis.shape[0] != half):
            raise ValueError("positions must be [n] or [axes, n], freq_axis one axis a frequency")
    st = LIB.splash_qkv_append(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _DTYPES[dt], n, *strides, hq, hkv, D,
        _data(q_weight), _data(k_weight), eps, _data(inv_freq), _data(freq_axis), 2 * half, int(interleaved),
        rope_scale, _data(positions) if half else None, axes, slots.data_ptr(), q_out.data_ptr(),
        k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), P,
        num_pages, _data(device_status), _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_qkv_append")


def splash_kv_gather(k_pages, v_pages, k_scales, v_scales, slots, k_out, v_out,
                     device_status=None, stream=None) -> None:
    """Dequantised cached rows: ``k_out`` / ``v_out`` float32 or bfloat16
    [n, Hkv, D]; rows with slot -1 are left as they were."""
    _tensors(k_out=k_out, k_pages=k_pages, v_pages=v_pages)
    dt = k_out.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError("k_out must be float32 or bfloat16")
    dev = _check_all(((k_scales, "k_scales", torch.float32, 3),
                      (v_scales, "v_scales", torch.float32, 3), (slots, "slots", torch.int32, 1),
                      (k_out, "k_out", dt, 3), (v_out, "v_out", dt, 3)), device_status)
    pool = num_pages, hkv, P, D = _pool_on(k_pages, v_pages, dev)
    n = slots.shape[0]
    if k_out.shape != (n, hkv, D) or v_out.shape != k_out.shape \
            or k_scales.shape != pool[:3] or v_scales.shape != pool[:3]:
        raise ValueError("shape mismatch between the rows, the slots and the pool")
    st = LIB.splash_kv_gather(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                              v_scales.data_ptr(), slots.data_ptr(), n, hkv, D, P, num_pages,
                              k_out.data_ptr(), v_out.data_ptr(), _DTYPES[dt],
                              _data(device_status), _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_kv_gather")


def splash_token_state_stride(vocab: int) -> int:
    return int(LIB.splash_token_state_stride(int(vocab)))


def alloc_token_state(num_seqs: int, vocab: int, device="cuda") -> torch.Tensor:
    """An empty token history: int16 [num_seqs, splash_token_state_stride(vocab)]."""
    stride = splash_token_state_stride(vocab)
    if stride == 0:
        raise ValueError("vocabulary out of range")
    return torch.zeros((num_seqs, stride), dtype=torch.int16, device=device)


def splash_token_state_add(tokens, q_offsets, state, vocab: int, accepted=None,
                           prompt: bool = False, reset: bool = False, device_status=None,
                           stream=None) -> None:
    """Count ``tokens`` (packed by ``q_offsets``) into the history; the first
    ``accepted[b] + 1`` of each sequence where ``accepted`` is given."""
    i32 = torch.int32
    dev = _check_all(((tokens, "tokens", i32, 1), (q_offsets, "q_offsets", i32, 1),
                      (state, "state", torch.int16, 2), (accepted, "accepted", i32, 1)), device_status)
    B = state.shape[0]
    if q_offsets.shape[0] != B + 1 or (accepted is not None and accepted.shape[0] != B):
        raise ValueError("shape mismatch between the offsets, accepted and the state")
    st = LIB.splash_token_state_add(tokens.data_ptr(), tokens.shape[0], q_offsets.data_ptr(), B,
                                    _data(accepted), state.data_ptr(), state.shape[1], int(vocab),
                                    int(prompt), int(reset), _data(device_status),
                                    _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_token_state_add")


def splash_choose_targets_workspace_size(num_rows: int, vocab: int) -> int:
    return int(LIB.splash_choose_targets_workspace_size(int(num_rows), int(vocab)))


def alloc_target_workspace(num_rows: int, vocab: int, device="cuda") -> torch.Tensor:
    """Workspace for splash_choose_targets on up to ``num_rows`` rows."""
    n = splash_choose_targets_workspace_size(num_rows, vocab)
    if n == 0:
        raise ValueError("invalid shape for the workspace size query")
    return torch.empty(n, dtype=torch.uint8, device=device)


def splash_choose_targets(logits, q_offsets, target_tokens, workspace, max_block_len: int,
                          block_tokens=None, state=None, repetition=None, presence=None,
                          frequency=None, bias_offsets=None, bias_ids=None, bias_values=None,
                          mask=None, mask_rows=None, out=None, device_status=None,
                          stream=None) -> None:
    """``logits``: float32, bfloat16 or float16 [n, vocab] with contiguous rows
    (a view of wider rows is fine); ``mask``: int32 [masks, >= ceil(vocab/32)];
    ``out``: float32 [n, vocab], possibly ``logits`` itself."""
    _tensors(logits=logits)
    f32, i32 = torch.float32, torch.int32
    dev = _check_all(((q_offsets, "q_offsets", i32, 1), (target_tokens, "target_tokens", i32, 1),
                      (workspace, "workspace", torch.uint8, 1),
                      (block_tokens, "block_tokens", i32, 1), (state, "state", torch.int16, 2),
                      (repetition, "repetition", f32, 1), (presence, "presence", f32, 1),
                      (frequency, "frequency", f32, 1), (bias_offsets, "bias_offsets", i32, 1),
                      (bias_ids, "bias_ids", i32, 1), (bias_values, "bias_values", f32, 1),
                      (mask, "mask", i32, 2), (mask_rows, "mask_rows", i32, 1)), device_status)
    dt = logits.dtype
    if dt not in _DTYPES or logits.dim() != 2 or logits.get_device() != dev:
        raise TypeError(f"logits must be a 2-D float32, bfloat16 or float16 tensor on cuda:{dev}")
    n, vocab = logits.shape
    if logits.stride(1) != 1 and vocab > 1:
        raise ValueError("the rows of logits must be contiguous")
    B = q_offsets.shape[0] - 1
    if B < 0 or target_tokens.shape[0] != n:
        raise ValueError("q_offsets has num_seqs + 1 entries, target_tokens one a row")
    for t, name in ((repetition, "repetition"), (presence, "presence"), (frequency, "frequency")):
        if t is not None and t.shape[0] != B:
            raise ValueError(f"{name} must have one value per sequence")
    if (repetition is not None or presence is not None or frequency is not None) \
            and (state is None or block_tokens is None):
        raise ValueError("penalties need the token history and the block's tokens")
    if state is not None and state.shape[0] != B or \
            block_tokens is not None and block_tokens.shape[0] != n:
        raise ValueError("shape mismatch between the state, the block's tokens and the rows")
    if (bias_offsets is None) != (bias_ids is None) or (bias_ids is None) != (bias_values is None):
        raise ValueError("biases are three tensors: offsets, ids and values")
    if bias_offsets is not None and (bias_offsets.shape[0] != B + 1
                                     or bias_values.shape != bias_ids.shape):
        raise ValueError("shape mismatch between the bias tensors")
    if mask_rows is not None and (mask is None or mask_rows.shape[0] != n):
        raise ValueError("mask_rows has one entry a row and needs mask")
    if out is not None and (not isinstance(out, torch.Tensor) or out.dtype is not f32 or out.get_device() != dev
                            or tuple(out.shape) != (n, vocab)
                            or (out.stride(1) != 1 and vocab > 1)):
        raise ValueError("out must be float32 [n, vocab] with contiguous rows")
    st = LIB.splash_choose_targets(
        logits.data_ptr(), _DTYPES[dt], max(logits.stride(0), vocab) if n < 2 else logits.stride(0),
        n, vocab, q_offsets.data_ptr(), B, int(max_block_len), _data(block_tokens), _data(state),
        0 if state is None else state.shape[1], _data(repetition), _data(presence),
        _data(frequency), _data(bias_offsets), _data(bias_ids), _data(bias_values),
        0 if bias_ids is None else bias_ids.shape[0], _data(mask),
        0 if mask is None else mask.shape[1], 0 if mask is None else mask.shape[0],
        _data(mask_rows), _data(out),
        0 if out is None else (max(out.stride(0), vocab) if n < 2 else out.stride(0)),
        target_tokens.data_ptr(), workspace.data_ptr(), workspace.numel(), _data(device_status),
        _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_choose_targets")


# ---------------------------------------------------------------------------
# Verification of a tree of drafts. A step's small calls are bound by their host
# time, most of it these checks: one pass that asks each tensor for its type,
# device, shape and layout, and the wording apart.
# ---------------------------------------------------------------------------
def _check_shapes(required, optional, device_status) -> int:
    """required, optional: (tensor, name, dtype, shape) of contiguous tensors on the
    current device, the optional ones possibly None. Returns the device index."""
    dev = torch.cuda.current_device()
    try:
        for t, _, dtype, shape in required:
            if t.dtype is not dtype or t.get_device() != dev or t.shape != shape \
                    or not t.is_contiguous():
                break
        else:
            for t, _, dtype, shape in optional:
                if t is not None and (t.dtype is not dtype or t.get_device() != dev
                                      or t.shape != shape or not t.is_contiguous()):
                    break
            else:
                if device_status is None:
                    return dev
    except AttributeError:
        pass
    for t, name, _, _ in required:               # the same with words
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    both = (*required, *optional)
    _check_all([(t, name, dtype, None) for t, name, dtype, _ in both], device_status)
    for t, name, _, shape in both:
        if t is not None and t.shape != shape:
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return dev


def splash_tree_masks(parents, q_offsets, masks, max_block_len: int, context_lens=None,
                      depths=None, positions=None, device_status=None, stream=None) -> None:
    """Ancestor bits ``masks`` (int32 [n, >= ceil(max_block_len / 32)]), ``depths``
    and ``positions`` (int32 [n]; the positions need ``context_lens``) of the nodes
    of every tree."""
    _tensors(parents=parents, q_offsets=q_offsets, masks=masks)
    i32 = torch.int32
    n, B = parents.numel(), q_offsets.numel() - 1
    words = masks.shape[-1]
    dev = _check_shapes(((parents, "parents", i32, (n,)), (q_offsets, "q_offsets", i32, (B + 1,)),
                         (masks, "masks", i32, (n, words))),
                        ((context_lens, "context_lens", i32, (B,)), (depths, "depths", i32, (n,)),
                         (positions, "positions", i32, (n,))), device_status)
    if B < 0:
        raise ValueError("q_offsets has num_seqs + 1 entries")
    if positions is not None and context_lens is None:
        raise ValueError("positions need context_lens")
    st = LIB.splash_tree_masks(parents.data_ptr(), n, q_offsets.data_ptr(), _data(context_lens), B,
                               int(max_block_len), masks.data_ptr(), words,
                               _data(depths), _data(positions), _data(device_status),
                               _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_tree_masks")


def splash_verify_attention_tree_workspace_size(num_seqs: int, num_q_tokens: int, num_q_heads: int,
                                                num_kv_heads: int, head_dim: int,
                                                max_block_len: int, ctas: int = 0) -> int:
    return int(LIB.splash_verify_attention_tree_workspace_size(
        num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, max_block_len, ctas))


def alloc_tree_workspace(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim,
                         max_block_len, device="cuda", ctas: int = 0) -> torch.Tensor:
    """Workspace for splash_verify_attention_tree."""
    n = splash_verify_attention_tree_workspace_size(num_seqs, num_q_tokens, num_q_heads,
                                                    num_kv_heads, head_dim, max_block_len, ctas)
    if n == 0:
        raise ValueError("invalid shape for the workspace size query")
    return torch.empty(n, dtype=torch.uint8, device=device)


def splash_verify_attention_tree(q, k_pages, v_pages, k_scales, v_scales, page_table,
                                 context_lens, block_lens, tree_masks, sm_scale: float,
                                 max_block_len: int, out, lse, workspace, device_status=None,
                                 stream=None, ctas: int = 0) -> None:
    """splash_verify_attention under the block masks ``tree_masks`` (int32
    [n, words], as splash_tree_masks writes them). The workspace from
    ``alloc_tree_workspace``."""
    _tensors(q=q, k_pages=k_pages, v_pages=v_pages, page_table=page_table,
             context_lens=context_lens, tree_masks=tree_masks, workspace=workspace)
    f32, i32, b16 = torch.float32, torch.int32, torch.bfloat16
    if q.dim() != 3 or page_table.dim() != 2 or tree_masks.dim() != 2 or k_pages.dim() != 4:
        raise ValueError("q has 3 dims, page_table and tree_masks 2, the pages 4")
    n, hq, d = qs = q.shape
    B, max_pages = context_lens.numel(), page_table.shape[1]
    words, room = tree_masks.shape[1], workspace.numel()
    num_pages, hkv, P, D = pool = k_pages.shape
    dev = _check_shapes(((q, "q", b16, qs), (out, "out", b16, qs), (lse, "lse", f32, (n, hq)),
                         (k_scales, "k_scales", f32, pool[:3]),
                         (v_scales, "v_scales", f32, pool[:3]),
                         (page_table, "page_table", i32, (B, max_pages)),
                         (context_lens, "context_lens", i32, (B,)),
                         (block_lens, "block_lens", i32, (B,)),
                         (tree_masks, "tree_masks", i32, (n, words)),
                         (workspace, "workspace", torch.uint8, (room,))), (), device_status)
    _pool_on(k_pages, v_pages, dev)
    if d != D or P != PAGE_SIZE:
        raise ValueError("shape mismatch between q and the pool")
    st = LIB.splash_verify_attention_tree(
        q.data_ptr(), n, k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
        v_scales.data_ptr(), page_table.data_ptr(), max_pages, context_lens.data_ptr(),
        block_lens.data_ptr(), tree_masks.data_ptr(), words, B, hq, hkv, D, P,
        num_pages, int(max_block_len), float(sm_scale), out.data_ptr(), lse.data_ptr(),
        workspace.data_ptr(), room, _data(device_status), _raw_stream(stream, dev),
        int(ctas))
    if st != 0:
        raise SplashError(st, "splash_verify_attention_tree")


def splash_accept_tree(block_tokens, parents, target_tokens, q_offsets, context_lens, accepted,
                       next_tokens, path_rows, path_tokens, max_block_len: int,
                       context_lens_out=None, device_status=None, stream=None) -> None:
    """The accepted path through every tree: its rows and tokens (``path_tokens``
    may be None), the accepted counts and next tokens. ``context_lens`` is advanced
    in place unless ``context_lens_out`` is given."""
    _tensors(block_tokens=block_tokens, context_lens=context_lens)
    ctx_out = context_lens if context_lens_out is None else context_lens_out
    i32 = torch.int32
    n, B = block_tokens.numel(), context_lens.numel()
    rows, seqs = (n,), (B,)
    dev = _check_shapes(((block_tokens, "block_tokens", i32, rows), (parents, "parents", i32, rows),
                         (target_tokens, "target_tokens", i32, rows),
                         (q_offsets, "q_offsets", i32, (B + 1,)),
                         (context_lens, "context_lens", i32, seqs),
                         (ctx_out, "context_lens_out", i32, seqs),
                         (accepted, "accepted", i32, seqs),
                         (next_tokens, "next_tokens", i32, seqs),
                         (path_rows, "path_rows", i32, rows)),
                        ((path_tokens, "path_tokens", i32, rows),), device_status)
    st = LIB.splash_accept_tree(
        block_tokens.data_ptr(), parents.data_ptr(), target_tokens.data_ptr(), n,
        q_offsets.data_ptr(), context_lens.data_ptr(), ctx_out.data_ptr(), accepted.data_ptr(),
        next_tokens.data_ptr(), path_rows.data_ptr(), _data(path_tokens), B, int(max_block_len),
        _data(device_status), _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_accept_tree")


def splash_kv_compact(k_pages, v_pages, k_scales, v_scales, slots, path_rows, q_offsets, accepted,
                      device_status=None, stream=None) -> None:
    """The cache rows of the accepted nodes moved to the block's first slots, in one
    pool or, with a leading layer axis on the pool's four tensors (``alloc_pool(...,
    num_layers=L)``), in every layer's."""
    _tensors(k_pages=k_pages, v_pages=v_pages, slots=slots, accepted=accepted)
    f32, i32 = torch.float32, torch.int32
    shape, strides = k_pages.shape, k_pages.stride()
    n, B = slots.numel(), accepted.numel()
    dev = _check_shapes(((k_scales, "k_scales", f32, shape[:-1]),
                         (v_scales, "v_scales", f32, shape[:-1]), (slots, "slots", i32, (n,)),
                         (path_rows, "path_rows", i32, (n,)),
                         (q_offsets, "q_offsets", i32, (B + 1,)),
                         (accepted, "accepted", i32, (B,))), (), device_status)
    layers, code_layer, scale_layer = 1, 0, 0
    if len(shape) == 5:
        layers, code_layer = shape[0], strides[0]
        num_pages, hkv, P, D = shape[1:]
        scale_layer = num_pages * hkv * P
        if layers == 0 or v_pages.shape != shape or v_pages.stride() != strides \
                or k_pages.dtype is not torch.int8 or v_pages.dtype is not torch.int8 \
                or strides[1:] != (hkv * 2 * P * D, 2 * P * D, D, 1) \
                or v_pages.data_ptr() != k_pages.data_ptr() + P * D \
                or k_pages.get_device() != dev:
            raise ValueError("k_pages and v_pages must be the halves of one pool per layer (see "
                             "alloc_pool) on the current device")
    else:
        num_pages, hkv, P, D = _pool_on(k_pages, v_pages, dev)
    if P != PAGE_SIZE:
        raise ValueError(f"pages of {PAGE_SIZE} slots, not {P}")
    st = LIB.splash_kv_compact(
        k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
        code_layer, scale_layer, layers, slots.data_ptr(), path_rows.data_ptr(), n,
        q_offsets.data_ptr(), accepted.data_ptr(), B, hkv, D, P, num_pages, _data(device_status),
        _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_kv_compact")


def splash_token_logprobs_workspace_size(num_out: int, vocab: int) -> int:
    return int(LIB.splash_token_logprobs_workspace_size(int(num_out), int(vocab)))


def alloc_logprobs_workspace(num_out: int, vocab: int, device="cuda") -> torch.Tensor:
    """Workspace for splash_token_logprobs of up to ``num_out`` rows."""
    n = splash_token_logprobs_workspace_size(num_out, vocab)
    if n == 0:
        raise ValueError("invalid shape for the workspace size query")
    return torch.empty(n, dtype=torch.uint8, device=device)


def splash_token_logprobs(logits, workspace, tokens=None, logprobs=None, entropy=None,
                          top_ids=None, top_logprobs=None, rows=None, device_status=None,
                          stream=None) -> None:
    """``logits``: float32, bfloat16 or float16 [n, vocab] with contiguous rows (a
    view of wider rows is fine). Outputs have one entry a row, or one per entry of
    ``rows`` (int32, -1: left as it was); ``tokens`` (int32 [n]) goes by the logits'
    rows. ``top_ids`` / ``top_logprobs``: int32 / float32 [outputs, k], k <= 32."""
    _tensors(logits=logits, workspace=workspace)
    f32, i32 = torch.float32, torch.int32
    dt = logits.dtype
    if dt not in _DTYPES or logits.dim() != 2:
        raise TypeError("logits must be a 2-D float32, bfloat16 or float16 tensor")
    if (tokens is None) != (logprobs is None) or (top_ids is None) != (top_logprobs is None):
        raise ValueError("tokens go with logprobs, top_ids with top_logprobs")
    if rows is not None:
        _tensors(rows=rows)
    if top_ids is not None:
        _tensors(top_ids=top_ids)
    n, vocab = logits.shape
    m = n if rows is None else rows.numel()
    top = 0 if top_ids is None else top_ids.shape[-1]
    room = workspace.numel()
    dev = _check_shapes(((workspace, "workspace", torch.uint8, (room,)),),
                        ((tokens, "tokens", i32, (n,)), (logprobs, "logprobs", f32, (m,)),
                         (entropy, "entropy", f32, (m,)), (top_ids, "top_ids", i32, (m, top)),
                         (top_logprobs, "top_logprobs", f32, (m, top)),
                         (rows, "rows", i32, (m,))), device_status)
    if logits.get_device() != dev:
        raise ValueError(f"logits is on {logits.device}, the current device is cuda:{dev}")
    pitch, step = logits.stride()
    if step != 1 and vocab > 1:
        raise ValueError("the rows of logits must be contiguous")
    st = LIB.splash_token_logprobs(
        logits.data_ptr(), _DTYPES[dt], max(pitch, vocab) if n < 2 else pitch,
        n, vocab, _data(rows), m, _data(tokens), _data(logprobs), _data(entropy),
        top, _data(top_ids), _data(top_logprobs),
        workspace.data_ptr(), room, _data(device_status), _raw_stream(stream, dev))
    if st != 0:
        raise SplashError(st, "splash_token_logprobs")
