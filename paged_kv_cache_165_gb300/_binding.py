"""ctypes binding of libpkv.so (the C ABI in include/pkv.h).

Argument marshalling only: each function checks that the torch tensors it is
given have the device, dtype, contiguity and shapes the C call expects, then
passes raw pointers, sizes and the current CUDA stream.  All computation runs in
the library's kernels; there is no fallback when the library is missing.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

from . import _build

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA = range(5)
PKV_F32, PKV_BF16, PKV_FP8_E4M3 = 0, 1, 2

DEVERR = {
    "slot": 1, "block": 2, "len": 4, "cu_seqlens": 8, "pair": 16, "timeout": 32, "layout": 64, "prefix": 128,
    "pool": 256,
}

_DTYPES = {torch.float32: PKV_F32, torch.bfloat16: PKV_BF16, torch.uint8: PKV_FP8_E4M3}


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pkv status {status}: {message}")
        self.status = status


_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded libpkv.so with argument types set.  Raises if it was never built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first with "
                           "paged_kv_cache_165_gb300._build.build() (needs nvcc)")
    L = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.pkv_status_string.argtypes = [I]
    L.pkv_status_string.restype = ctypes.c_char_p
    L.pkv_last_error.argtypes = []
    L.pkv_last_error.restype = ctypes.c_char_p
    L.pkv_version.argtypes = []
    L.pkv_version.restype = I
    L.pkv_kv_append.argtypes = [P, P, P, P, I, P, I, I, I, I, I, P]
    L.pkv_kv_append.restype = I
    L.pkv_kv_block_copy.argtypes = [P, P, I, P, I, I, I, I, I, P]
    L.pkv_kv_block_copy.restype = I
    L.pkv_decode_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    L.pkv_decode_workspace_bytes.restype = Z
    L.pkv_paged_attention_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I, I, I]
    L.pkv_paged_attention_workspace_bytes.restype = Z
    L.pkv_paged_attention.argtypes = [P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, I, I, F, I, I, P,
                                      Z, P]
    L.pkv_paged_attention.restype = I
    L.pkv_paged_attention_kernel_launches.argtypes = [I, I, I, I, I, I, I, I, I, I, I, I]
    L.pkv_paged_attention_kernel_launches.restype = I
    L.pkv_kv_append_fp8.argtypes = [P, P, I, P, P, P, P, P, I, I, I, I, I, P]
    L.pkv_kv_append_fp8.restype = I
    L.pkv_paged_decode_attention_fp8.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I,
                                                 P, Z, P]
    L.pkv_paged_decode_attention_fp8.restype = I
    L.pkv_decode_kernel_launches.argtypes = [I, I, I, I, I, I, I, I, I]
    L.pkv_decode_kernel_launches.restype = I
    L.pkv_paged_decode_attention.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, F, I, P,
                                             Z, P]
    L.pkv_paged_decode_attention.restype = I
    L.pkv_decode_step.argtypes = [P, P, P, P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, F, I, P, Z, P]
    L.pkv_decode_step.restype = I
    L.pkv_decode_step_kernel_launches.argtypes = [I, I, I, I, I, I, I, I, I]
    L.pkv_decode_step_kernel_launches.restype = I
    L.pkv_decode_step_fp8.argtypes = [P, P, P, P, P, I, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, Z, P]
    L.pkv_decode_step_fp8.restype = I
    L.pkv_decode_step_fp8_kernel_launches.argtypes = [I, I, I, I, I, I, I, I, I]
    L.pkv_decode_step_fp8_kernel_launches.restype = I
    L.pkv_paged_decode_attention_noalloc.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I,
                                                     F, I, P]
    L.pkv_paged_decode_attention_noalloc.restype = I
    L.pkv_decode_step_shared_prefix.argtypes = [P, P, P, P, P, P, P, P, I, P, P, P, P, P, I, I, I, I, I, I, I, I,
                                                I, I, I, F, I, P, Z, P]
    L.pkv_decode_step_shared_prefix.restype = I
    L.pkv_decode_step_shared_prefix_workspace_bytes.argtypes = [I] * 11
    L.pkv_decode_step_shared_prefix_workspace_bytes.restype = Z
    L.pkv_decode_step_shared_prefix_kernel_launches.argtypes = [I] * 13
    L.pkv_decode_step_shared_prefix_kernel_launches.restype = I
    L.pkv_q4_row_bytes.argtypes = [I, I]
    L.pkv_q4_row_bytes.restype = I
    for name in ("pkv_kv_append_q4", "pkv_kv_gather_q4"):
        getattr(L, name).argtypes = [P, P, I, P, P, P, I, I, I, I, I, I, P]
        getattr(L, name).restype = I
    L.pkv_paged_attention_q4_workspace_bytes.argtypes = [I] * 11
    L.pkv_paged_attention_q4_workspace_bytes.restype = Z
    L.pkv_paged_attention_q4.argtypes = [P] * 8 + [I] * 10 + [F, I, I, P, Z, P]
    L.pkv_paged_attention_q4.restype = I
    L.pkv_decode_step_q4.argtypes = [P, P, P, P, P, I, P, P, P, P, P] + [I] * 8 + [F, I, I, P, Z, P]
    L.pkv_decode_step_q4.restype = I
    L.pkv_block_tables_extend_workspace_bytes.argtypes = [I, I]
    L.pkv_block_tables_extend_workspace_bytes.restype = Z
    L.pkv_block_tables_extend.argtypes = [P] * 9 + [I] * 5 + [P, Z, P]
    L.pkv_block_tables_extend.restype = I
    L.pkv_block_tables_extend_step.argtypes = [P] * 10 + [I] * 5 + [P, Z, P]
    L.pkv_block_tables_extend_step.restype = I
    L.pkv_block_tables_release_workspace_bytes.argtypes = [I]
    L.pkv_block_tables_release_workspace_bytes.restype = Z
    L.pkv_block_tables_release.argtypes = [P] * 6 + [I] * 3 + [P, Z, P]
    L.pkv_block_tables_release.restype = I
    L.pkv_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, I, I, P, P]
    L.pkv_selftest_bounded_wait.restype = I
    L.pkv_prefill_attention.argtypes = [P, P, P, P, P, I, P, I, I, I, I, I, I, F, P, P, P, I, I, P]
    L.pkv_prefill_attention.restype = I
    L.pkv_get_device_error.argtypes = [ctypes.POINTER(I), P]
    L.pkv_get_device_error.restype = I
    _lib = L
    return L


def header_functions() -> list:
    """Names of the functions include/pkv.h declares."""
    with open(os.path.join(_build.INCLUDE, "pkv.h")) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pkv_[a-z_0-9]+)\s*\(", text)))


# ------------------------------------------------------------------ helpers

def _check(status: int) -> None:
    if status != PKV_OK:
        raise PkvError(status, lib().pkv_last_error().decode(errors="replace"))


# The current stream's handle without the Stream object around it, which costs microseconds to make.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, here=None) -> int:   # here: the current device, where it is known
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if here is None else here)
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _bytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8


def _cuda(name, t, dtype=None):
    if type(t) is torch.Tensor and t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current_device() -> int:
    try:
        return _raw_device()
    except (RuntimeError, AssertionError):   # no driver: no tensor is there either
        return -2


def _ready(here, tensors) -> bool:
    """Contiguous tensors of device `here`, all of them (None: left out)?  Eager decode steps are short
    enough for the checks' cost to show: this is their common outcome, _refuse says what is wrong."""
    for t in tensors:
        if t is not None and (t.get_device() != here or not t.is_contiguous()):
            return False
    return True


_OPTIONAL = ("lse", "cu_q", "first_block", "step_slots", "workspace")


def _refuse(what, here, **tensors) -> None:
    """The error of whatever _ready or a type found wrong.  tensors: name=(tensor, its type or None)."""
    for name, (t, dtype) in tensors.items():
        if t is not None or name not in _OPTIONAL:
            _cuda(name, t, dtype)
            if t.get_device() != here:   # the kernels run on the current device
                raise ValueError(f"{what}: {name} is on device {t.get_device()}, the current one is {here}")


def _dtype(t) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported element type {t.dtype} (fp32, bf16 or uint8 E4M3 codes)")
    return _DTYPES[t.dtype]


# --------------------------------------------------------------------- ABI

def kv_append(k_new, v_new, k_cache, v_cache, slot_mapping, stream=None) -> None:
    """k_new/v_new [T][Hkv][d] -> cache slots slot_mapping[t] (int64, <0 skipped)."""
    _cuda("k_cache", k_cache)
    dt = _dtype(k_cache)
    _cuda("v_cache", v_cache, k_cache.dtype)
    _cuda("k_new", k_new, k_cache.dtype)
    _cuda("v_new", v_new, k_cache.dtype)
    _cuda("slot_mapping", slot_mapping, torch.int64)
    NB, Hkv, bs, d = k_cache.shape
    T = k_new.shape[0]
    if tuple(k_new.shape) != (T, Hkv, d) or tuple(v_new.shape) != (T, Hkv, d) or slot_mapping.numel() != T:
        raise ValueError("kv_append: shapes do not match [T][Hkv][d] / [T]")
    _check(lib().pkv_kv_append(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), dt,
                               _ptr(slot_mapping), T, Hkv, d, bs, NB, _stream(stream)))


def kv_append_fp8(k_new, v_new, k_codes, v_codes, k_scale, v_scale, slot_mapping, stream=None) -> None:
    """Quantise k_new/v_new [T][Hkv][d] (bf16 or fp32) into E4M3 codes [NB][Hkv][bs][d]
    (uint8) and fp32 row scales [NB][Hkv][bs] at slot_mapping[t] (int64, <0 skipped)."""
    _cuda("k_new", k_new)
    new_dt = _dtype(k_new)
    _cuda("v_new", v_new, k_new.dtype)
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
        _cuda(name, t, torch.uint8)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _cuda(name, t, torch.float32)
    _cuda("slot_mapping", slot_mapping, torch.int64)
    NB, Hkv, bs, d = k_codes.shape
    T = k_new.shape[0]
    if tuple(k_new.shape) != (T, Hkv, d) or tuple(v_new.shape) != (T, Hkv, d) or \
            tuple(v_codes.shape) != (NB, Hkv, bs, d) or tuple(k_scale.shape) != (NB, Hkv, bs) or \
            tuple(v_scale.shape) != (NB, Hkv, bs) or slot_mapping.numel() != T:
        raise ValueError("kv_append_fp8: shapes do not match")
    _check(lib().pkv_kv_append_fp8(_ptr(k_new), _ptr(v_new), new_dt, _ptr(k_codes), _ptr(v_codes),
                                   _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping), T, Hkv, d, bs, NB,
                                   _stream(stream)))


def paged_decode_attention_fp8(out, q, k_codes, v_codes, k_scale, v_scale, block_table, context_lens,
                               scale, window=0, lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """Decode attention (one query per sequence) over an E4M3 cache with row scales."""
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
        _cuda(name, t, torch.uint8)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _cuda(name, t, torch.float32)
    _cuda("q", q, torch.float32)
    _cuda("out", out, torch.float32)
    _cuda("block_table", block_table, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    NB, Hkv, bs, d = k_codes.shape
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d) or block_table.dim() != 2 or \
            block_table.shape[0] != B or context_lens.numel() != B or \
            (lse is not None and lse.numel() != B * Hq):
        raise ValueError("paged_decode_attention_fp8: shapes do not match")
    ws_bytes = 0
    if workspace is not None:
        _cuda("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().pkv_paged_decode_attention_fp8(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
        _ptr(block_table), _ptr(context_lens), B, Hq, Hkv, d, bs, block_table.shape[1], NB, float(scale),
        int(window), int(num_splits), _ptr(workspace), ws_bytes, _stream(stream)))


def kv_block_copy(k_cache, v_cache, pairs, stream=None) -> None:
    """Copy whole blocks: for each (src, dst) row of int32 pairs [n][2]."""
    _cuda("k_cache", k_cache)
    dt = _dtype(k_cache)
    _cuda("v_cache", v_cache, k_cache.dtype)
    _cuda("pairs", pairs, torch.int32)
    NB, Hkv, bs, d = k_cache.shape
    n = pairs.numel() // 2
    _check(lib().pkv_kv_block_copy(_ptr(k_cache), _ptr(v_cache), dt, _ptr(pairs), n, Hkv, d, bs,
                                   NB, _stream(stream)))


def decode_workspace_bytes(B, Hq, Hkv, d, bs, MBS, num_splits=0) -> int:
    return int(lib().pkv_decode_workspace_bytes(B, Hq, Hkv, d, bs, MBS, num_splits))


def decode_kernel_launches(B, Hq, Hkv, d, bs, MBS, NB, dtype, num_splits=0) -> int:
    """Kernels one paged_decode_attention call with these sizes enqueues (-1: rejected)."""
    dt = _DTYPES[dtype]
    return int(lib().pkv_decode_kernel_launches(B, Hq, Hkv, d, bs, MBS, NB, dt, num_splits))


def paged_decode_attention(out, q, k_cache, v_cache, block_table, context_lens, scale, lse=None,
                           num_splits=0, workspace=None, stream=None) -> None:
    """out [B][Hq][d] fp32 = attention of q [B][Hq][d] fp32 over the paged cache."""
    _cuda("k_cache", k_cache)
    dt = _dtype(k_cache)
    _cuda("v_cache", v_cache, k_cache.dtype)
    _cuda("q", q, torch.float32)
    _cuda("out", out, torch.float32)
    _cuda("block_table", block_table, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    NB, Hkv, bs, d = k_cache.shape
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d) or block_table.dim() != 2 or \
            block_table.shape[0] != B or context_lens.numel() != B or \
            (lse is not None and lse.numel() != B * Hq):
        raise ValueError("paged_decode_attention: shapes do not match")
    MBS = block_table.shape[1]
    ws_bytes = 0
    if workspace is not None:
        _cuda("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().pkv_paged_decode_attention(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table),
        _ptr(context_lens), B, Hq, Hkv, d, bs, MBS, NB, float(scale), int(num_splits),
        _ptr(workspace), ws_bytes, _stream(stream)))


def decode_step(out, q, k_new, v_new, slot_mapping, k_cache, v_cache, block_table, context_lens, scale,
                lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """One decode step: k_new/v_new [B][Hkv][d] (row b = sequence b's new token) go to
    slot_mapping[b] (int64, < 0: none), then out [B][Hq][d] fp32 = attention of q over the
    cache (context_lens count the new tokens).  One launch where the library fuses them."""
    _cuda("k_cache", k_cache)
    dt = _dtype(k_cache)
    _cuda("v_cache", v_cache, k_cache.dtype)
    _cuda("k_new", k_new, k_cache.dtype)
    _cuda("v_new", v_new, k_cache.dtype)
    _cuda("slot_mapping", slot_mapping, torch.int64)
    _cuda("q", q, torch.float32)
    _cuda("out", out, torch.float32)
    _cuda("block_table", block_table, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    NB, Hkv, bs, d = k_cache.shape
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d) or tuple(k_new.shape) != (B, Hkv, d) or \
            tuple(v_new.shape) != (B, Hkv, d) or slot_mapping.numel() != B or block_table.dim() != 2 or \
            block_table.shape[0] != B or context_lens.numel() != B or \
            (lse is not None and lse.numel() != B * Hq):
        raise ValueError("decode_step: shapes do not match")
    ws_bytes = 0
    if workspace is not None:
        _cuda("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().pkv_decode_step(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache),
        _ptr(v_cache), dt, _ptr(block_table), _ptr(context_lens), B, Hq, Hkv, d, bs, block_table.shape[1],
        NB, float(scale), int(num_splits), _ptr(workspace), ws_bytes, _stream(stream)))


def decode_step_shared_prefix(out, q, k_new, v_new, slot_mapping, k_cache, v_cache, block_table, context_lens,
                              scale, groups, lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """decode_step where the batch rows of each group in ``groups`` (a PrefixGroups on the
    device) share a prefix of physical blocks: the same results, with each group's prefix
    read once."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_new", k_new), ("v_new", v_new)):
        _cuda(name, t, k_cache.dtype)
    dt = _dtype(k_cache)
    _cuda("slot_mapping", slot_mapping, torch.int64)
    _cuda("q", q, torch.float32)
    _cuda("out", out, torch.float32)
    _cuda("block_table", block_table, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    for name in ("prefix_tokens", "group_start", "group_seqs"):
        _cuda(name, getattr(groups, name), torch.int32)
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    NB, Hkv, bs, d = k_cache.shape
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d) or tuple(k_new.shape) != (B, Hkv, d) or \
            tuple(v_new.shape) != (B, Hkv, d) or slot_mapping.numel() != B or block_table.dim() != 2 or \
            block_table.shape[0] != B or context_lens.numel() != B or groups.prefix_tokens.numel() != B or \
            (lse is not None and lse.numel() != B * Hq):
        raise ValueError("decode_step_shared_prefix: shapes do not match")
    ws_bytes = 0
    if workspace is not None:
        _cuda("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().pkv_decode_step_shared_prefix(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache),
        _ptr(v_cache), dt, _ptr(block_table), _ptr(context_lens), _ptr(groups.prefix_tokens),
        _ptr(groups.group_start), _ptr(groups.group_seqs), groups.n_groups, groups.n_members,
        groups.max_group_size, groups.max_prefix_tokens, B, Hq, Hkv, d, bs, block_table.shape[1], NB,
        float(scale), int(num_splits), _ptr(workspace), ws_bytes, _stream(stream)))


def decode_step_shared_prefix_workspace_bytes(B, Hq, Hkv, d, bs, MBS, groups, num_splits=0) -> int:
    return int(lib().pkv_decode_step_shared_prefix_workspace_bytes(
        B, Hq, Hkv, d, bs, MBS, int(num_splits), groups.n_groups, groups.n_members, groups.max_group_size,
        groups.max_prefix_tokens))


def decode_step_shared_prefix_kernel_launches(B, Hq, Hkv, d, bs, MBS, NB, dtype, groups, num_splits=0) -> int:
    return int(lib().pkv_decode_step_shared_prefix_kernel_launches(
        B, Hq, Hkv, d, bs, MBS, NB, _DTYPES[dtype], int(num_splits), groups.n_groups, groups.n_members,
        groups.max_group_size, groups.max_prefix_tokens))


def decode_step_kernel_launches(B, Hq, Hkv, d, bs, MBS, NB, dtype, num_splits=0) -> int:
    """Kernels one decode_step call with these sizes enqueues (-1: rejected)."""
    return int(lib().pkv_decode_step_kernel_launches(B, Hq, Hkv, d, bs, MBS, NB, _DTYPES[dtype],
                                                     int(num_splits)))


def paged_attention_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, bs, MBS, window=0, num_splits=0) -> int:
    return int(lib().pkv_paged_attention_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, bs, MBS, window,
                                                         num_splits))


def paged_attention_kernel_launches(B, Tq, max_q, Hq, Hkv, d, bs, MBS, NB, dtype, window=0,
                                    num_splits=0) -> int:
    """Kernels one paged_attention call with these sizes enqueues (-1: rejected)."""
    return int(lib().pkv_paged_attention_kernel_launches(B, Tq, max_q, Hq, Hkv, d, bs, MBS, NB,
                                                         _DTYPES[dtype], window, num_splits))


def paged_attention(out, q, k_cache, v_cache, block_table, context_lens, scale, cu_q=None, max_q=1,
                    window=0, lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """Queries at the end of each cached sequence (causal, optional sliding window).

    q, out [Tq][Hq][d] fp32; cu_q int32 [B+1] (None: one query per sequence)."""
    _cuda("k_cache", k_cache)
    dt = _dtype(k_cache)
    _cuda("v_cache", v_cache, k_cache.dtype)
    _cuda("q", q, torch.float32)
    _cuda("out", out, torch.float32)
    _cuda("block_table", block_table, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    if cu_q is not None:
        _cuda("cu_q", cu_q, torch.int32)
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    NB, Hkv, bs, d = k_cache.shape
    Tq, Hq, dq = q.shape
    B = context_lens.numel()
    if dq != d or tuple(out.shape) != (Tq, Hq, d) or block_table.dim() != 2 or \
            block_table.shape[0] != B or (cu_q is not None and cu_q.numel() != B + 1) or \
            (cu_q is None and Tq != B) or (lse is not None and lse.numel() != Tq * Hq):
        raise ValueError("paged_attention: shapes do not match")
    ws_bytes = 0
    if workspace is not None:
        _cuda("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().pkv_paged_attention(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table),
        _ptr(context_lens), _ptr(cu_q), B, Tq, int(max_q), Hq, Hkv, d, bs, block_table.shape[1], NB,
        float(scale), int(window), int(num_splits), _ptr(workspace), ws_bytes, _stream(stream)))


def paged_decode_attention_noalloc(out, q, k_cache, v_cache, block_table, context_lens, scale,
                                   lse=None, num_splits=0, stream=None) -> None:
    """paged_decode_attention with the library's built-in split-K scratch (no workspace)."""
    _cuda("k_cache", k_cache)
    dt = _dtype(k_cache)
    _cuda("v_cache", v_cache, k_cache.dtype)
    _cuda("q", q, torch.float32)
    _cuda("out", out, torch.float32)
    _cuda("block_table", block_table, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    NB, Hkv, bs, d = k_cache.shape
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d) or block_table.dim() != 2 or \
            block_table.shape[0] != B or context_lens.numel() != B or \
            (lse is not None and lse.numel() != B * Hq):
        raise ValueError("paged_decode_attention_noalloc: shapes do not match")
    _check(lib().pkv_paged_decode_attention_noalloc(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table),
        _ptr(context_lens), B, Hq, Hkv, d, bs, block_table.shape[1], NB, float(scale),
        int(num_splits), _stream(stream)))


def prefill_attention(out, q, k, v, cu_seqlens, max_seqlen, scale, lse=None, k_cache=None,
                      v_cache=None, slot_mapping=None, stream=None) -> None:
    """Varlen causal attention of packed q [T][Hq][d], k/v [T][Hkv][d]; optional cache write."""
    _cuda("q", q)
    dt = _dtype(q)
    _cuda("k", k, q.dtype)
    _cuda("v", v, q.dtype)
    _cuda("out", out, torch.float32)
    _cuda("cu_seqlens", cu_seqlens, torch.int32)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if tuple(k.shape) != (T, Hkv, d) or tuple(v.shape) != (T, Hkv, d) or tuple(out.shape) != (T, Hq, d):
        raise ValueError("prefill_attention: shapes do not match")
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    bs = NB = 0
    if slot_mapping is not None:
        _cuda("slot_mapping", slot_mapping, torch.int64)
        _cuda("k_cache", k_cache, q.dtype)
        _cuda("v_cache", v_cache, q.dtype)
        NB, _, bs, _ = k_cache.shape
    _check(lib().pkv_prefill_attention(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k), _ptr(v), dt, _ptr(cu_seqlens), B, T,
        int(max_seqlen), Hq, Hkv, d, float(scale), _ptr(k_cache), _ptr(v_cache),
        _ptr(slot_mapping), bs, NB, _stream(stream)))


def selftest_bounded_wait(limit_ns, blocks, hold_tmem=True, gave_up=None, stream=None) -> None:
    """Run the kernels' bounded-wait failure path on purpose: `blocks` blocks wait on an
    mbarrier no copy completes, give up after limit_ns and tear down (PKV_DEVERR_TIMEOUT).
    gave_up: optional int32 device tensor of one element counting the threads that gave up."""
    if gave_up is not None:
        _cuda("gave_up", gave_up, torch.int32)
    _check(lib().pkv_selftest_bounded_wait(int(limit_ns), int(blocks), 1 if hold_tmem else 0, _ptr(gave_up),
                                           _stream(stream)))


def get_device_error(stream=None) -> int:
    """Synchronise the stream; return and clear the device error bits."""
    code = ctypes.c_int(0)
    _check(lib().pkv_get_device_error(ctypes.byref(code), _stream(stream)))
    return code.value


def decode_step_fp8(out, q, k_new, v_new, slot_mapping, k_codes, v_codes, k_scale, v_scale, block_table,
                    context_lens, scale, lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """decode_step over an E4M3 cache: k_new/v_new [B][Hkv][d] (bf16 or fp32) are quantised
    into codes [NB][Hkv][bs][d] (uint8) and row scales [NB][Hkv][bs] (fp32) at
    slot_mapping[b], then out [B][Hq][d] fp32 = attention of q over the cache."""
    _cuda("k_new", k_new)
    new_dt = _dtype(k_new)
    _cuda("v_new", v_new, k_new.dtype)
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
        _cuda(name, t, torch.uint8)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _cuda(name, t, torch.float32)
    _cuda("slot_mapping", slot_mapping, torch.int64)
    _cuda("q", q, torch.float32)
    _cuda("out", out, torch.float32)
    _cuda("block_table", block_table, torch.int32)
    _cuda("context_lens", context_lens, torch.int32)
    if lse is not None:
        _cuda("lse", lse, torch.float32)
    NB, Hkv, bs, d = k_codes.shape
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d) or tuple(k_new.shape) != (B, Hkv, d) or \
            tuple(v_new.shape) != (B, Hkv, d) or tuple(v_codes.shape) != (NB, Hkv, bs, d) or \
            tuple(k_scale.shape) != (NB, Hkv, bs) or tuple(v_scale.shape) != (NB, Hkv, bs) or \
            slot_mapping.numel() != B or block_table.dim() != 2 or block_table.shape[0] != B or \
            context_lens.numel() != B or (lse is not None and lse.numel() != B * Hq):
        raise ValueError("decode_step_fp8: shapes do not match")
    ws_bytes = 0
    if workspace is not None:
        _cuda("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().pkv_decode_step_fp8(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_new), _ptr(v_new), new_dt, _ptr(slot_mapping), _ptr(k_codes),
        _ptr(v_codes), _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(context_lens), B, Hq, Hkv, d, bs,
        block_table.shape[1], NB, float(scale), int(num_splits), _ptr(workspace), ws_bytes, _stream(stream)))


def decode_step_fp8_kernel_launches(B, Hq, Hkv, d, bs, MBS, NB, new_dtype=torch.bfloat16, num_splits=0) -> int:
    """Kernels one decode_step_fp8 call with these sizes enqueues (-1: rejected)."""
    return int(lib().pkv_decode_step_fp8_kernel_launches(B, Hq, Hkv, d, bs, MBS, NB, _DTYPES[new_dtype],
                                                         int(num_splits)))


# ----------------------------------------------------------------- 4-bit cache

@functools.lru_cache(maxsize=None)
def q4_row_bytes(d, group) -> int:
    """Bytes of one row of a 4-bit cache (codes and its share of the page's parameters): the
    last dimension of k_cache and v_cache, uint8 [NB][Hkv][bs][q4_row_bytes(d, group)]."""
    n = int(lib().pkv_q4_row_bytes(int(d), int(group)))
    if n < 0:
        raise ValueError(f"q4_row_bytes: d={d} group={group} (group 32, 64 or 128, d a multiple of it, d <= 256)")
    return n


def _q4_caches(what, k_cache, v_cache, d, group):
    shape = k_cache.shape
    if len(shape) != 4 or shape != v_cache.shape or shape[3] != q4_row_bytes(d, group):
        raise ValueError(f"{what}: the caches must be [NB][Hkv][bs][{q4_row_bytes(d, group)}] (q4_row_bytes of d={d}, "
                         f"group={group}), got {tuple(shape)} and {tuple(v_cache.shape)}")
    return shape


def _q4_rows(what, fn, k_rows, v_rows, k_cache, v_cache, slot_mapping, group, stream):
    here = _current_device()
    try:
        ok = (_ready(here, (k_rows, v_rows, k_cache, v_cache, slot_mapping)) and k_rows.dtype is v_rows.dtype and
              k_cache.dtype is _U8 and v_cache.dtype is _U8 and slot_mapping.dtype is _I64)
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(what, here, k_rows=(k_rows, None), v_rows=(v_rows, getattr(k_rows, "dtype", None)), k_cache=(k_cache, _U8),
                v_cache=(v_cache, _U8), slot_mapping=(slot_mapping, _I64))
    dt = _dtype(k_rows)
    rows = k_rows.shape
    if len(rows) != 3:
        raise ValueError(f"{what}: rows must be [T][Hkv][d]")
    T, H, d = rows
    NB, Hkv, bs, _ = _q4_caches(what, k_cache, v_cache, d, group)
    if H != Hkv or v_rows.shape != rows or slot_mapping.numel() != T:
        raise ValueError(f"{what}: shapes do not match [T][Hkv][d] / [T]")
    status = fn(k_rows.data_ptr(), v_rows.data_ptr(), dt, k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), T,
                Hkv, d, int(group), bs, NB, _stream(stream, here))
    if status:
        _check(status)


def kv_append_q4(k_new, v_new, k_cache, v_cache, slot_mapping, group, stream=None) -> None:
    """Quantise k_new/v_new [T][Hkv][d] (bf16 or fp32) into a 4-bit cache, uint8
    [NB][Hkv][bs][q4_row_bytes(d, group)], at slot_mapping[t] (int64, <0 skipped)."""
    _q4_rows("kv_append_q4", lib().pkv_kv_append_q4, k_new, v_new, k_cache, v_cache, slot_mapping, group, stream)


def kv_gather_q4(k_out, v_out, k_cache, v_cache, slot_mapping, group, stream=None) -> None:
    """k_out/v_out [T][Hkv][d] (bf16 or fp32) = the values of the rows at slot_mapping[t]
    (int64; rows of zeros for negative slots)."""
    _q4_rows("kv_gather_q4", lib().pkv_kv_gather_q4, k_out, v_out, k_cache, v_cache, slot_mapping, group, stream)


def paged_attention_q4_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, group, bs, MBS, window=0, num_splits=0) -> int:
    return int(lib().pkv_paged_attention_q4_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, group, bs, MBS, window,
                                                            num_splits))


def _q4_attend_sizes(what, out, q, k_cache, v_cache, block_table, context_lens, group, lse):
    rows = q.shape
    if len(rows) != 3:
        raise ValueError(f"{what}: q must be [rows][Hq][d]")
    Tq, Hq, d = rows
    B = context_lens.numel()
    NB, Hkv, bs, _ = _q4_caches(what, k_cache, v_cache, d, group)
    table = block_table.shape
    if out.shape != rows or len(table) != 2 or table[0] != B or (lse is not None and lse.numel() != Tq * Hq):
        raise ValueError(f"{what}: shapes do not match")
    return B, Tq, Hq, Hkv, d, bs, NB, table[1]


def paged_attention_q4(out, q, k_cache, v_cache, block_table, context_lens, scale, group, cu_q=None, max_q=1,
                       window=0, lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """paged_attention over a 4-bit cache: q, out [Tq][Hq][d] fp32, the newest rows of every
    sequence (cu_q int32 [B+1]; None: one row per sequence), causal, optional window."""
    what, here = "paged_attention_q4", _current_device()
    try:
        ok = (_ready(here, (out, q, k_cache, v_cache, block_table, context_lens, lse, cu_q, workspace)) and q.dtype is _F32 and
              out.dtype is _F32 and k_cache.dtype is _U8 and v_cache.dtype is _U8 and block_table.dtype is _I32 and
              context_lens.dtype is _I32 and (lse is None or lse.dtype is _F32) and (cu_q is None or cu_q.dtype is _I32))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(what, here, q=(q, _F32), out=(out, _F32), k_cache=(k_cache, _U8), v_cache=(v_cache, _U8),
                block_table=(block_table, _I32), context_lens=(context_lens, _I32), lse=(lse, _F32), cu_q=(cu_q, _I32),
                workspace=(workspace, None))
    B, Tq, Hq, Hkv, d, bs, NB, MBS = _q4_attend_sizes(what, out, q, k_cache, v_cache, block_table, context_lens, group, lse)
    if cu_q.numel() != B + 1 if cu_q is not None else Tq != B:
        raise ValueError("paged_attention_q4: shapes do not match")
    status = lib().pkv_paged_attention_q4(
        out.data_ptr(), _ptr(lse), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
        context_lens.data_ptr(), _ptr(cu_q), B, Tq, int(max_q), Hq, Hkv, d, int(group), bs, MBS, NB, float(scale), int(window),
        int(num_splits), _ptr(workspace), _bytes(workspace), _stream(stream, here))
    if status:
        _check(status)


def decode_step_q4(out, q, k_new, v_new, slot_mapping, k_cache, v_cache, block_table, context_lens, scale, group,
                   window=0, lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """decode_step over a 4-bit cache: k_new/v_new [B][Hkv][d] (bf16 or fp32) are quantised into
    slot_mapping[b] (int64, < 0: none), then out [B][Hq][d] fp32 = attention of q over the cache."""
    what, here = "decode_step_q4", _current_device()
    try:
        ok = (_ready(here, (out, q, k_new, v_new, slot_mapping, k_cache, v_cache, block_table, context_lens, lse, workspace)) and
              q.dtype is _F32 and out.dtype is _F32 and k_new.dtype is v_new.dtype and slot_mapping.dtype is _I64 and
              k_cache.dtype is _U8 and v_cache.dtype is _U8 and block_table.dtype is _I32 and context_lens.dtype is _I32 and
              (lse is None or lse.dtype is _F32))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(what, here, q=(q, _F32), out=(out, _F32), k_new=(k_new, None), v_new=(v_new, getattr(k_new, "dtype", None)),
                slot_mapping=(slot_mapping, _I64), k_cache=(k_cache, _U8), v_cache=(v_cache, _U8),
                block_table=(block_table, _I32), context_lens=(context_lens, _I32), lse=(lse, _F32), workspace=(workspace, None))
    B, Tq, Hq, Hkv, d, bs, NB, MBS = _q4_attend_sizes(what, out, q, k_cache, v_cache, block_table, context_lens, group, lse)
    new_dt, new = _dtype(k_new), k_new.shape
    if Tq != B or new != (B, Hkv, d) or v_new.shape != new or slot_mapping.numel() != B:
        raise ValueError("decode_step_q4: shapes do not match")
    status = lib().pkv_decode_step_q4(
        out.data_ptr(), _ptr(lse), q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), new_dt, slot_mapping.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(), B, Hq, Hkv, d, int(group), bs,
        MBS, NB, float(scale), int(window), int(num_splits), _ptr(workspace), _bytes(workspace), _stream(stream, here))
    if status:
        _check(status)


# ---------------------------------------------------------------- block tables

def block_tables_extend_workspace_bytes(B, T) -> int:
    return int(lib().pkv_block_tables_extend_workspace_bytes(int(B), int(T)))


def block_tables_release_workspace_bytes(B) -> int:
    return int(lib().pkv_block_tables_release_workspace_bytes(int(B)))


def block_tables_extend(block_table, context_lens, new_tokens, free_list, free_count, context_lens_out, cu_new,
                        slot_mapping, free_count_out, bs, workspace=None, stream=None, step_slots=None) -> None:
    """Blocks, table entries and slots for new_tokens[b] more tokens of every row (see pkv.h).

    block_table int32 [B][MBS]; context_lens, new_tokens, context_lens_out int32 [B]; free_list
    int32 [NB]; free_count, free_count_out int32 [1]; cu_new int32 [B+1]; slot_mapping int64 [T]
    (the new tokens row after row; entries past them become -1).  step_slots: int64 [B], the
    slot of each row's last new token, -1 where it got none (what decode_step* take; None: left out).
    The *_out tensors may be their inputs."""
    what, here = "block_tables_extend", _current_device()
    ints = (block_table, context_lens, new_tokens, free_list, free_count, context_lens_out, cu_new, free_count_out)
    try:
        ok = (_ready(here, (*ints, slot_mapping, step_slots, workspace)) and all([t.dtype is _I32 for t in ints]) and
              slot_mapping.dtype is _I64 and (step_slots is None or step_slots.dtype is _I64))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(what, here, block_table=(block_table, _I32), context_lens=(context_lens, _I32), new_tokens=(new_tokens, _I32),
                free_list=(free_list, _I32), free_count=(free_count, _I32), context_lens_out=(context_lens_out, _I32),
                cu_new=(cu_new, _I32), free_count_out=(free_count_out, _I32), slot_mapping=(slot_mapping, _I64),
                step_slots=(step_slots, _I64), workspace=(workspace, None))
    table = block_table.shape
    if len(table) != 2:
        raise ValueError("block_tables_extend: block_table must be [B][MBS]")
    B, MBS = table
    if context_lens.numel() != B or new_tokens.numel() != B or context_lens_out.numel() != B or \
            cu_new.numel() != B + 1 or free_count.numel() != 1 or free_count_out.numel() != 1 or \
            (step_slots is not None and step_slots.numel() != B):
        raise ValueError("block_tables_extend: shapes do not match")
    tables = (block_table.data_ptr(), context_lens.data_ptr(), new_tokens.data_ptr(), free_list.data_ptr(), free_count.data_ptr(),
              context_lens_out.data_ptr(), cu_new.data_ptr(), slot_mapping.data_ptr())
    sizes = (free_count_out.data_ptr(), B, slot_mapping.numel(), MBS, int(bs), free_list.numel(), _ptr(workspace),
             _bytes(workspace), _stream(stream, here))
    if step_slots is None:
        status = lib().pkv_block_tables_extend(*tables, *sizes)
    else:
        status = lib().pkv_block_tables_extend_step(*tables, step_slots.data_ptr(), *sizes)
    if status:
        _check(status)


def block_tables_release(block_table, first_block, end_block, free_list, free_count, free_count_out, workspace=None,
                         stream=None) -> None:
    """Logical blocks [first_block[b], end_block[b]) of every row (int32 [B]; first_block None: 0)
    back to the free list, their table entries -1 (see pkv.h)."""
    what, here = "block_tables_release", _current_device()
    ints = (block_table, end_block, free_list, free_count, free_count_out)
    try:
        ok = (_ready(here, (*ints, first_block, workspace)) and all([t.dtype is _I32 for t in ints]) and
              (first_block is None or first_block.dtype is _I32))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(what, here, block_table=(block_table, _I32), end_block=(end_block, _I32), free_list=(free_list, _I32),
                free_count=(free_count, _I32), free_count_out=(free_count_out, _I32), first_block=(first_block, _I32),
                workspace=(workspace, None))
    table = block_table.shape
    if len(table) != 2:
        raise ValueError("block_tables_release: block_table must be [B][MBS]")
    B, MBS = table
    if end_block.numel() != B or (first_block is not None and first_block.numel() != B) or free_count.numel() != 1 or \
            free_count_out.numel() != 1:
        raise ValueError("block_tables_release: shapes do not match")
    status = lib().pkv_block_tables_release(
        block_table.data_ptr(), _ptr(first_block), end_block.data_ptr(), free_list.data_ptr(), free_count.data_ptr(),
        free_count_out.data_ptr(), B, MBS, free_list.numel(), _ptr(workspace), _bytes(workspace), _stream(stream, here))
    if status:
        _check(status)
