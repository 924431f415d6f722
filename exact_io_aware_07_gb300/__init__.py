"""FlashAttention forward on one GB300: Python binding of the C-ABI library ``libfa_gb300.so``.

The binding only marshals arguments: it checks tensor dtypes, shapes and
devices, then passes raw device pointers and the current CUDA stream to the
C entry points declared in ``include/fa.h``.  Every step of the attention
computation runs in the library's sm_103a kernel; there is no other path.  If
the library has not been built, importing works but the first call raises.

Entry points (same names as the C ABI):
    fa_fwd(q, k, v, o, lse, causal, scale, stream=None)
    fa_fwd_gqa(q, k, v, o, lse, causal, scale, stream=None)
    fa_fwd_paged(q, k_pages, v_pages, block_table, o, lse, causal, scale, stream=None)
    fa_fwd_fp8(q8, k8, v8, o, lse, causal, scale, descales, workspace, stream=None)
    fa_fwd_splitkv(q, k, v, o, lse, causal, scale, num_splits, workspace, stream=None)
    fa_fwd_splitkv_noalloc(q, k, v, o, lse, causal, scale, num_splits, stream=None)
    fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, causal, scale, workspace, stream=None)
    fa_page_plan(ctx_lens, new_lens, free_pages, free_head, block_table, seq_lens, cu_new, slot_map,
                 free_head_out, num_pages, stream=None)
    fa_kv_append(k_new, v_new, slot_map, k_pages, v_pages, stream=None)
    fa_fwd_prefix_paged(q, k_pages, v_pages, prefix_table, prefix_len, block_table, seq_lens, cu_new, max_new,
                        o, lse, causal, scale, workspace=None, stream=None)
    fa_fwd_splitkv_workspace_bytes, fa_fwd_splitkv_count, fa_fwd_fp8_workspace_bytes, fa_bwd_workspace_bytes,
    fa_fwd_prefix_paged_workspace_bytes
    fa_status_string(code), fa_device_status(stream=None), fa_selftest_wait_timeout(us, stream=None)
    fa_fwd_launch_shape(B, H, T, d, causal, num_sms), fa_ex2_rate(stream=None), fa_version()
and the convenience wrappers ``attention``, ``attention_gqa``, ``attention_splitkv``,
``attention_bwd``, ``page_plan`` and ``attention_prefix_paged`` that allocate their
outputs (and workspaces) with PyTorch.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

from ._build import build, lib_path  # noqa: F401

__all__ = [
    "FAError", "fa_fwd", "fa_fwd_splitkv", "fa_fwd_splitkv_noalloc", "fa_fwd_splitkv_workspace_bytes",
    "fa_fwd_splitkv_count", "fa_status_string", "fa_device_status", "FA_NOALLOC_SCRATCH_BYTES",
    "fa_fwd_launch_shape", "fa_selftest_wait_timeout", "fa_ex2_rate", "fa_version",
    "attention", "attention_splitkv", "load_library", "STATUS", "FA_MAX_SPLITS",
    "fa_page_plan", "page_plan", "fa_kv_append", "fa_fwd_prefix_paged", "fa_fwd_prefix_paged_workspace_bytes",
    "attention_prefix_paged", "PAGE",
]

STATUS = {
    0: "FA_OK", 1: "FA_ERR_NULL_PTR", 2: "FA_ERR_MISALIGNED", 3: "FA_ERR_BAD_SHAPE",
    4: "FA_ERR_UNSUPPORTED_HEAD_DIM", 5: "FA_ERR_BAD_SCALE", 6: "FA_ERR_NO_DEVICE_SUPPORT",
    7: "FA_ERR_LAUNCH", 8: "FA_ERR_DEVICE_TIMEOUT", 9: "FA_ERR_BAD_ARG", 10: "FA_ERR_BAD_POINTER",
    11: "FA_ERR_ALIAS", 12: "FA_ERR_CUDA", 13: "FA_ERR_WORKSPACE", 14: "FA_ERR_BAD_PAGE",
    15: "FA_ERR_BAD_LENGTH", 16: "FA_ERR_NO_PAGES",
}
FA_MAX_SPLITS = 256
EXPORTED = ["fa_fwd", "fa_fwd_gqa", "fa_fwd_paged", "fa_fwd_fp8", "fa_fwd_fp8_workspace_bytes", "fa_bwd",
            "fa_bwd_workspace_bytes", "fa_fwd_splitkv", "fa_fwd_splitkv_noalloc", "fa_fwd_splitkv_workspace_bytes",
            "fa_fwd_splitkv_count", "fa_status_string", "fa_device_status", "fa_fwd_launch_shape", "fa_selftest_wait_timeout", "fa_ex2_rate",
            "fa_version", "fa_page_plan", "fa_kv_append", "fa_fwd_prefix_paged", "fa_fwd_prefix_paged_workspace_bytes"]
PAGE = 128  # keys per page of a paged cache
FA_NOALLOC_SCRATCH_BYTES = 32 << 20


class FAError(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, code: int, where: str):
        self.code = code
        self.name = STATUS.get(code, str(code))
        super().__init__(f"{where}: {self.name} ({fa_status_string(code)})")


_LIB = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Loads the built library (once).  Raises if it is missing: there is no fallback."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"attention library not built ({path}); run exact_io_aware_07_gb300.build()")
    lib = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    lib.fa_fwd_gqa.restype = i
    lib.fa_fwd_paged.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, f, f, f, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_fwd_fp8_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_fwd_fp8_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, f, vp, ctypes.c_size_t, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i]
    lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_device_status.argtypes = [vp, ctypes.POINTER(i)]
    lib.fa_device_status.restype = i
    lib.fa_fwd_launch_shape.argtypes = [i, i, i, i, i, i] + [ctypes.POINTER(i)] * 3
    lib.fa_fwd_launch_shape.restype = i
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_splitkv_noalloc.restype = i
    lib.fa_fwd_splitkv_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_fwd_splitkv_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_splitkv_count.argtypes = [i, i, i, i, i, i]
    lib.fa_fwd_splitkv_count.restype = i
    lib.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
    lib.fa_selftest_wait_timeout.restype = i
    lib.fa_ex2_rate.argtypes = [ctypes.POINTER(ctypes.c_double), vp]
    lib.fa_ex2_rate.restype = i
    ll = ctypes.c_longlong
    lib.fa_page_plan.argtypes = [vp] * 9 + [i] * 5 + [vp]
    lib.fa_page_plan.restype = i
    lib.fa_kv_append.argtypes = [vp] * 5 + [i, i, i, ll, ll, i, vp]
    lib.fa_kv_append.restype = i
    lib.fa_fwd_prefix_paged.argtypes = [vp] * 9 + [i] * 8 + [f, i, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_prefix_paged.restype = i
    lib.fa_fwd_prefix_paged_workspace_bytes.argtypes = [i] * 5
    lib.fa_fwd_prefix_paged_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_version.argtypes = []
    lib.fa_version.restype = ctypes.c_char_p
    if path == lib_path():
        _LIB = lib
    return lib


def fa_status_string(code: int) -> str:
    return load_library().fa_status_string(int(code)).decode()


def fa_version() -> str:
    return load_library().fa_version().decode()


def fa_fwd_launch_shape(B: int, H: int, T: int, d: int, causal: bool, num_sms: int):
    """(grid, threads, dynamic smem bytes) of the launch ``fa_fwd`` makes for these sizes."""
    g, t, s = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    code = load_library().fa_fwd_launch_shape(B, H, T, d, int(causal), num_sms,
                                              ctypes.byref(g), ctypes.byref(t), ctypes.byref(s))
    if code:
        raise FAError(code, "fa_fwd_launch_shape")
    return g.value, t.value, s.value


def _stream_handle(stream):
    import torch

    if stream is None:  # the raw handle: making a Stream object of it takes 2.5 us
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_stream(stream):
    """Context in which PyTorch allocates and fills tensors on ``stream`` (an int handle or a Stream; None: the current
    one), so that a kernel there finds them in order and their memory is reused in order."""
    import torch

    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def fa_device_status(stream=None) -> int:
    """Reads and clears the device status word (0 = FA_OK, 8 = a wait ran out)."""
    out = ctypes.c_int()
    code = load_library().fa_device_status(ctypes.c_void_p(_stream_handle(stream)), ctypes.byref(out))
    if code:
        raise FAError(code, "fa_device_status")
    return out.value


def fa_selftest_wait_timeout(timeout_us: int, stream=None) -> None:
    """Enqueues the bounded-wait self-test kernel (see include/fa.h); read the outcome with fa_device_status."""
    code = load_library().fa_selftest_wait_timeout(int(timeout_us), ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_selftest_wait_timeout")


def fa_ex2_rate(stream=None) -> float:
    """ex2.approx operations per second of the current device (a short probe; synchronous)."""
    out = ctypes.c_double(0.0)
    code = load_library().fa_ex2_rate(ctypes.byref(out), ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_ex2_rate")
    return float(out.value)


def fa_fwd(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """O, LSE = attention(Q, K, V) into caller-owned tensors.

    q, k, v, o: bf16 CUDA tensors (B, H, T, d), contiguous; lse: fp32 (B, H, T).
    Enqueued on ``stream`` (default: PyTorch's current stream); not synchronised.
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 (B, H, T, d) tensor")
    if not (q.shape == k.shape == v.shape == o.shape):
        raise ValueError("q, k, v and o must have the same shape")
    B, H, T, d = q.shape
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 (B, H, T) tensor")
    lib = load_library()
    code = lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                      B, H, T, d, int(bool(causal)), float(scale), ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_fwd")


def fa_fwd_gqa(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """Grouped K/V heads: q, o (B, H, T, d) and k, v (B, Hkv, T, d) bf16, H a multiple of Hkv;
    query head h reads K/V head h // (H // Hkv).  lse: fp32 (B, H, T)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 4-D tensor")
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    if tuple(o.shape) != (B, H, T, d) or tuple(k.shape) != (B, Hkv, T, d) or k.shape != v.shape:
        raise ValueError("q, o must be (B, H, T, d) and k, v (B, Hkv, T, d)")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 (B, H, T) tensor")
    code = load_library().fa_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                     B, H, Hkv, T, d, int(bool(causal)), float(scale),
                                     ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_fwd_gqa")


def attention_gqa(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Allocates O and LSE and runs ``fa_fwd_gqa``; ``scale`` defaults to 1/sqrt(d)."""
    import torch

    B, H, T, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    fa_fwd_gqa(q, k, v, o, lse, causal, scale, stream)
    return o, lse


def fa_fwd_paged(q, k_pages, v_pages, block_table, o, lse, causal: bool, scale: float, stream=None) -> None:
    """Paged K/V: k_pages, v_pages (num_pages, Hkv, 128, d) bf16; block_table (B, max_pages) int32 on the
    device; q, o (B, H, T, d) bf16; lse (B, H, T) fp32.  Key t of batch entry b is row t % 128 of page
    block_table[b, t // 128]."""
    import torch

    for name, t in (("q", q), ("k_pages", k_pages), ("v_pages", v_pages), ("o", o)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 4-D tensor")
    B, H, T, d = q.shape
    num_pages, Hkv, page, dk = k_pages.shape
    if page != 128 or dk != d or v_pages.shape != k_pages.shape or tuple(o.shape) != (B, H, T, d):
        raise ValueError("pages must be (num_pages, Hkv, 128, d), like q's d")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 (B, max_pages) tensor")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 (B, H, T) tensor")
    code = load_library().fa_fwd_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                       o.data_ptr(), lse.data_ptr(), B, H, Hkv, T, d, int(bool(causal)),
                                       float(scale), num_pages, block_table.shape[1],
                                       ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_fwd_paged")


def _check_int(name, t, shape, int32):
    if t.dtype is not int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}")


def _check_pools(k_pages, v_pages):
    """(num_pages, Hkv, d) of two page pools."""
    import torch

    shape, bf16 = k_pages.shape, torch.bfloat16
    if not (k_pages.dtype is bf16 and v_pages.dtype is bf16 and len(shape) == 4 and shape[2] == PAGE
            and v_pages.shape == shape and k_pages.is_contiguous() and v_pages.is_contiguous()):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.dtype is not bf16 or t.dim() != 4 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous bf16 4-D tensor")
        raise ValueError(f"pages must be (num_pages, Hkv, {PAGE}, d)")
    return shape[0], shape[1], shape[3]


def fa_page_plan(ctx_lens, new_lens, free_pages, free_head, block_table, seq_lens, cu_new, slot_map, free_head_out,
                 num_pages: int, stream=None) -> None:
    """Block table and slot map of a step, from the requests' lengths (all int32 CUDA tensors).

    ctx_lens, new_lens: (B), the tokens each request holds and adds; free_pages (any number of page numbers) and
    free_head (1), how many of them are taken.  Updates block_table (B, max_pages) in place; writes seq_lens (B),
    cu_new (B + 1), slot_map (max_tokens; -1 behind the last new token) and free_head_out (1).
    """
    import torch

    if block_table.dim() != 2 or slot_map.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("block_table must be (B, max_pages), slot_map and free_pages one-dimensional")
    B, max_pages = table = block_table.shape
    tokens, free = slot_map.shape, free_pages.shape
    i32, batch, one = torch.int32, (B,), (1,)
    # (written out: nine calls would take a fourth of a small plan's time)
    if not (ctx_lens.dtype is i32 and new_lens.dtype is i32 and free_pages.dtype is i32 and free_head.dtype is i32
            and block_table.dtype is i32 and seq_lens.dtype is i32 and cu_new.dtype is i32 and slot_map.dtype is i32
            and free_head_out.dtype is i32 and ctx_lens.shape == batch and new_lens.shape == batch
            and free_head.shape == one and seq_lens.shape == batch and cu_new.shape == (B + 1,)
            and free_head_out.shape == one and ctx_lens.is_contiguous() and new_lens.is_contiguous()
            and free_pages.is_contiguous() and block_table.is_contiguous() and seq_lens.is_contiguous()
            and cu_new.is_contiguous() and slot_map.is_contiguous()):
        for name, t, shape in (("ctx_lens", ctx_lens, batch), ("new_lens", new_lens, batch),
                               ("free_pages", free_pages, free), ("free_head", free_head, one),
                               ("block_table", block_table, table), ("seq_lens", seq_lens, batch),
                               ("cu_new", cu_new, (B + 1,)), ("slot_map", slot_map, tokens),
                               ("free_head_out", free_head_out, one)):
            _check_int(name, t, shape, i32)
    code = load_library().fa_page_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
                                       free_head.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                                       cu_new.data_ptr(), slot_map.data_ptr(), free_head_out.data_ptr(), B, max_pages,
                                       int(num_pages), free[0], tokens[0], _stream_handle(stream))
    if code:
        raise FAError(code, "fa_page_plan")


def page_plan(ctx_lens, new_lens, free_pages, free_head, block_table, max_tokens: int, num_pages: int, stream=None):
    """Allocates and returns (seq_lens, cu_new, slot_map, free_head_out) of ``fa_page_plan``, which updates
    ``block_table`` in place; ``max_tokens`` is the length of the slot map."""
    import torch

    B = ctx_lens.shape[0]
    with _on_stream(stream):
        seq, cu, slots, head = (torch.empty(n, dtype=torch.int32, device=ctx_lens.device)
                                for n in (B, B + 1, max_tokens, 1))
    fa_page_plan(ctx_lens, new_lens, free_pages, free_head, block_table, seq, cu, slots, head, num_pages, stream)
    return seq, cu, slots, head


def fa_kv_append(k_new, v_new, slot_map, k_pages, v_pages, stream=None) -> None:
    """Writes new keys and values (N, Hkv, d) bf16 into the page pools (num_pages, Hkv, 128, d) by slot_map (N) int32
    (negative: skipped).  The heads of a token must be contiguous; tokens may be any multiple of 8 elements apart."""
    import torch

    num_pages, Hkv, d = _check_pools(k_pages, v_pages)
    N = slot_map.shape[0] if slot_map.dim() == 1 else -1
    _check_int("slot_map", slot_map, (N,), torch.int32)
    shape, strides = (N, Hkv, d), []
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.dtype is not torch.bfloat16 or t.shape != shape:
            raise ValueError(f"{name} must be a bf16 (N, Hkv, d) tensor, like the pages and slot_map")
        token, head, column = t.stride()
        if column != 1 or (Hkv > 1 and head != d):
            raise ValueError(f"{name} must have contiguous heads")
        strides.append(token)
    code = load_library().fa_kv_append(k_new.data_ptr(), v_new.data_ptr(), slot_map.data_ptr(), k_pages.data_ptr(),
                                       v_pages.data_ptr(), N, Hkv, d, strides[0], strides[1], num_pages,
                                       _stream_handle(stream))
    if code:
        raise FAError(code, "fa_kv_append")


def fa_fwd_prefix_paged_workspace_bytes(N: int, B: int, H: int, Hkv: int, d: int) -> int:
    return int(load_library().fa_fwd_prefix_paged_workspace_bytes(N, B, H, Hkv, d))


def fa_fwd_prefix_paged(q, k_pages, v_pages, prefix_table, prefix_len: int, block_table, seq_lens, cu_new,
                        max_new: int, o, lse, causal: bool, scale: float, workspace=None, stream=None) -> None:
    """New tokens' attention over a shared prefix and each request's own pages.

    q, o: bf16 (N, H, d), request b's tokens at rows cu_new[b] .. cu_new[b + 1] - 1; k_pages, v_pages: bf16
    (num_pages, Hkv, 128, d); prefix_table: int32, the pages of the ``prefix_len`` keys all requests share (None when
    there are none); block_table (B, max_pages), seq_lens (B: own keys with the new ones) and cu_new (B + 1): int32;
    ``max_new``: the largest number of new tokens of a request; lse: fp32 (N, H).  ``workspace``: a CUDA tensor of at
    least ``fa_fwd_prefix_paged_workspace_bytes`` bytes (allocated here when None).
    """
    import torch

    num_pages, Hkv, d = _check_pools(k_pages, v_pages)
    rows, table, i32, bf16 = q.shape, block_table.shape, torch.int32, torch.bfloat16
    if not (q.dtype is bf16 and o.dtype is bf16 and len(rows) == 3 and rows[2] == d and o.shape == rows
            and q.is_contiguous() and o.is_contiguous()):
        for name, t in (("q", q), ("o", o)):
            if t.dtype is not bf16 or t.dim() != 3 or t.shape[2] != d or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous bf16 (N, H, d) tensor")
        raise ValueError("q and o must have the same shape")
    N, H, _ = rows
    if lse.dtype is not torch.float32 or lse.shape != rows[:2] or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 (N, H) tensor")
    if len(table) != 2:
        raise ValueError("block_table must be (B, max_pages)")
    B, max_pages = table
    if not (block_table.dtype is i32 and seq_lens.dtype is i32 and cu_new.dtype is i32 and seq_lens.shape == (B,)
            and cu_new.shape == (B + 1,) and block_table.is_contiguous() and seq_lens.is_contiguous()
            and cu_new.is_contiguous()):
        _check_int("block_table", block_table, table, i32)
        _check_int("seq_lens", seq_lens, (B,), i32)
        _check_int("cu_new", cu_new, (B + 1,), i32)
    if prefix_table is not None:
        _check_int("prefix_table", prefix_table, (prefix_table.numel(),), i32)
    if prefix_len > 0 and (prefix_table is None or prefix_table.numel() * PAGE < prefix_len):
        raise ValueError("prefix_table must hold ceil(prefix_len / 128) pages")
    if workspace is None:
        with _on_stream(stream):
            workspace = torch.empty(max(1, fa_fwd_prefix_paged_workspace_bytes(N, B, H, Hkv, d)), dtype=torch.uint8,
                                    device=q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    code = load_library().fa_fwd_prefix_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                              prefix_table.data_ptr() if prefix_len > 0 else None,
                                              block_table.data_ptr(), seq_lens.data_ptr(), cu_new.data_ptr(),
                                              o.data_ptr(), lse.data_ptr(), N, B, H, Hkv, d, int(prefix_len),
                                              int(max_new), int(bool(causal)), float(scale), num_pages, max_pages,
                                              workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if code:
        raise FAError(code, "fa_fwd_prefix_paged")


def attention_prefix_paged(q, k_pages, v_pages, prefix_table, prefix_len: int, block_table, seq_lens, cu_new,
                           max_new: int, causal: bool = True, scale: float | None = None, stream=None):
    """Allocates O, LSE and the workspace and runs ``fa_fwd_prefix_paged``; ``scale`` defaults to 1/sqrt(d).  Rows
    behind the last request's come back as zeros with an LSE of -infinity."""
    import torch

    N, H, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _on_stream(stream):
        o = torch.zeros_like(q)
        lse = torch.full((N, H), float("-inf"), dtype=torch.float32, device=q.device)
    fa_fwd_prefix_paged(q, k_pages, v_pages, prefix_table, prefix_len, block_table, seq_lens, cu_new, max_new, o, lse,
                        causal, scale, None, stream)
    return o, lse


def fa_fwd_fp8_workspace_bytes(B: int, H: int, T: int, d: int) -> int:
    return int(load_library().fa_fwd_fp8_workspace_bytes(B, H, T, d))


def fa_fwd_fp8(q, k, v, o, lse, causal: bool, scale: float, descales=(1.0, 1.0, 1.0), workspace=None,
               stream=None) -> None:
    """e4m3 Q, K, V (uint8 CUDA tensors (B, H, T, 128) holding the bytes) with per-tensor scales
    ``descales`` = (q, k, v); O bf16 (B, H, T, 128), LSE fp32 (B, H, T).  ``workspace``: a CUDA tensor
    of at least ``fa_fwd_fp8_workspace_bytes`` bytes (allocated here when None)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.uint8 or t.dim() != 4 or not t.is_contiguous() or t.shape != q.shape:
            raise ValueError(f"{name} must be a contiguous uint8 (B, H, T, d) tensor of e4m3 bytes")
    B, H, T, d = q.shape
    if o.dtype != torch.bfloat16 or tuple(o.shape) != (B, H, T, d) or not o.is_contiguous():
        raise ValueError("o must be a contiguous bf16 (B, H, T, d) tensor")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 (B, H, T) tensor")
    if workspace is None:
        workspace = torch.empty(max(1, fa_fwd_fp8_workspace_bytes(B, H, T, d)), dtype=torch.uint8, device=q.device)
    nbytes = workspace.numel() * workspace.element_size()
    qs, ks, vs = (float(x) for x in descales)
    code = load_library().fa_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                     B, H, T, d, int(bool(causal)), float(scale), qs, ks, vs,
                                     workspace.data_ptr(), nbytes, ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_fwd_fp8")


def fa_bwd_workspace_bytes(B: int, H: int, T: int) -> int:
    return int(load_library().fa_bwd_workspace_bytes(B, H, T))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, causal: bool, scale: float, workspace, stream=None) -> None:
    """dQ, dK, dV of sum(dO * O) into caller-owned bf16 tensors (all (B, H, T, d), contiguous).

    ``o`` and ``lse`` are what ``fa_fwd`` returned for (q, k, v, causal, scale);
    ``workspace`` is a CUDA tensor of at least ``fa_bwd_workspace_bytes(B, H, T)`` bytes.
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous() or t.shape != q.shape:
            raise ValueError(f"{name} must be a contiguous bf16 tensor shaped like q")
    B, H, T, d = q.shape
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 (B, H, T) tensor")
    nbytes = workspace.numel() * workspace.element_size()
    code = load_library().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, T, d,
                                 int(bool(causal)), float(scale), workspace.data_ptr(), nbytes,
                                 ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_bwd")


def attention_bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, stream=None):
    """Allocates dQ, dK, dV and the workspace and runs ``fa_bwd``; ``scale`` defaults to 1/sqrt(d)."""
    import torch

    B, H, T, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(fa_bwd_workspace_bytes(B, H, T), dtype=torch.uint8, device=q.device)
    fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, causal, scale, ws, stream)
    return dq, dk, dv


def attention(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Allocates O (bf16) and LSE (fp32) and runs ``fa_fwd``; ``scale`` defaults to 1/sqrt(d)."""
    import torch

    B, H, T, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, causal, scale, stream)
    return o, lse


def fa_fwd_splitkv_count(B: int, H: int, T: int, d: int, causal: bool, num_splits: int) -> int:
    """Key ranges ``fa_fwd_splitkv`` would use (``num_splits`` 0: the library's choice); -1 if invalid."""
    return int(load_library().fa_fwd_splitkv_count(B, H, T, d, int(bool(causal)), num_splits))


def fa_fwd_splitkv_workspace_bytes(B: int, H: int, T: int, d: int, num_splits: int) -> int:
    """Bytes of scratch ``fa_fwd_splitkv`` needs (0 for invalid sizes; ``num_splits`` 0: the automatic choice)."""
    return int(load_library().fa_fwd_splitkv_workspace_bytes(B, H, T, d, num_splits))


def _check_qkv_o_lse(q, k, v, o, lse):
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 (B, H, T, d) tensor")
    if not (q.shape == k.shape == v.shape == o.shape):
        raise ValueError("q, k, v and o must have the same shape")
    B, H, T, d = q.shape
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 (B, H, T) tensor")
    return B, H, T, d


def fa_fwd_splitkv(q, k, v, o, lse, causal: bool, scale: float, num_splits: int, workspace, stream=None) -> None:
    """Split-KV attention into caller-owned tensors; ``workspace`` is a CUDA tensor used as scratch."""
    B, H, T, d = _check_qkv_o_lse(q, k, v, o, lse)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    code = load_library().fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                         B, H, T, d, int(bool(causal)), float(scale), int(num_splits),
                                         workspace.data_ptr(), nbytes, ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_fwd_splitkv")


def attention_splitkv(q, k, v, causal: bool = False, num_splits: int = 0, scale: float | None = None, stream=None):
    """Allocates O, LSE and the split workspace and runs ``fa_fwd_splitkv`` (``num_splits`` 0: chosen by the library)."""
    import torch

    B, H, T, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    ws = torch.empty(fa_fwd_splitkv_workspace_bytes(B, H, T, d, num_splits), dtype=torch.uint8, device=q.device)
    fa_fwd_splitkv(q, k, v, o, lse, causal, scale, num_splits, ws, stream)
    return o, lse


def fa_fwd_splitkv_noalloc(q, k, v, o, lse, causal: bool, scale: float, num_splits: int, stream=None) -> None:
    """Split-KV attention with the library's fixed device scratch (no workspace, no allocation).

    For callers that cannot allocate device memory while running; see the
    declaration in include/fa.h for the size limit and the sharing rules.
    """
    B, H, T, d = _check_qkv_o_lse(q, k, v, o, lse)
    code = load_library().fa_fwd_splitkv_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                                 lse.data_ptr(), B, H, T, d, int(bool(causal)), float(scale),
                                                 int(num_splits), ctypes.c_void_p(_stream_handle(stream)))
    if code:
        raise FAError(code, "fa_fwd_splitkv_noalloc")
