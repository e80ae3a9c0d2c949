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
import platform
import re

import torch

from . import _build

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA = range(5)
PKV_F32, PKV_BF16, PKV_FP8_E4M3 = 0, 1, 2

DEVERR = {
    "slot": 1, "block": 2, "len": 4, "cu_seqlens": 8, "pair": 16, "timeout": 32, "layout": 64, "prefix": 128,
    "pool": 256, "probs": 512,
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
    if platform.machine() not in ("x86_64", "aarch64"):
        raise RuntimeError(f"the binding passes arguments as x86-64 and aarch64 do; this machine is {platform.machine()}")
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
    L.pkv_block_tables_share_workspace_bytes.argtypes = [I, I, I]
    L.pkv_block_tables_share_workspace_bytes.restype = Z
    # The whole numbers of the calls of a decode step are declared as pointers, whose conversion takes half as long: an
    # argument of 32 bits is the lower half of a 64-bit register or stack slot on both of x86-64 and aarch64 (lib() refuses
    # other machines).
    N = P
    L.pkv_block_tables_fork.argtypes = [P] * 11 + [N] * 4 + [P, N, P]
    L.pkv_block_tables_fork.restype = I
    L.pkv_block_tables_compact.argtypes = [P] * 9 + [N] * 4 + [P, N, P]
    L.pkv_block_tables_compact.restype = I
    L.pkv_kv_block_copy_counted.argtypes = [P, P, N, P, N, P, N, N, N, N, P]
    L.pkv_kv_block_copy_counted.restype = I
    D = ctypes.c_double
    L.pkv_rope_turns.argtypes = [P, I, D, I, D, D, D, D]
    L.pkv_rope_turns.restype = I
    L.pkv_rope_append.argtypes = [P, N, P, P, P, N, N, N, N, P, P, N, N, F, P, P, P] + [N] * 6 + [P]
    L.pkv_rope_append.restype = I
    L.pkv_rope.argtypes = [P, N, P, P, P, N, N, N, P, P, N, N, F, N, N, N, N, N, P]
    L.pkv_rope.restype = I
    L.pkv_verify_drafts.argtypes = [P, P, P, P, N, N, N, P, P, P, P, P, N, N, N, P]
    L.pkv_verify_drafts.restype = I
    L.pkv_paged_attention_sinks_workspace_bytes.argtypes = [I] * 11
    L.pkv_paged_attention_sinks_workspace_bytes.restype = Z
    L.pkv_paged_attention_sinks.argtypes = [P, P, P, P, P, N, P, P, P] + [N] * 9 + [F, N, N, N, P, N, P]
    L.pkv_paged_attention_sinks.restype = I
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


_OPTIONAL = ("lse", "cu_q", "first_block", "step_slots", "workspace", "parents", "held", "draft_probs", "context_lens_out")


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


def kv_block_copy(k_cache, v_cache, pairs, stream=None, count=None) -> None:
    """Copy whole blocks: for each (src, dst) row of int32 pairs [n][2].  count: int32 [1] on the
    device, the number of leading pairs to copy (pkv_kv_block_copy_counted)."""
    if count is not None:
        here = _current_device()
        try:
            ok = _ready(here, (k_cache, v_cache, pairs, count)) and pairs.dtype is _I32 and count.dtype is _I32 and \
                v_cache.dtype is k_cache.dtype
        except AttributeError:   # not a tensor
            ok = False
        if not ok:
            _refuse("kv_block_copy", here, k_cache=(k_cache, None), v_cache=(v_cache, getattr(k_cache, "dtype", None)),
                    pairs=(pairs, _I32), count=(count, _I32))
        shape = k_cache.shape
        if len(shape) != 4 or v_cache.shape != shape or count.numel() != 1:
            raise ValueError("kv_block_copy: shapes do not match")
        NB, Hkv, bs, d = shape
        status = lib().pkv_kv_block_copy_counted(k_cache.data_ptr(), v_cache.data_ptr(), _dtype(k_cache), pairs.data_ptr(),
                                                 pairs.numel() // 2, count.data_ptr(), Hkv, d, bs, NB, _stream(stream, here))
        if status:
            _check(status)
        return
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


def block_tables_share_workspace_bytes(B, MBS, NB) -> int:
    return int(lib().pkv_block_tables_share_workspace_bytes(int(B), int(MBS), int(NB)))


def _share_refuse(what, here, workspace, optional, **required) -> None:
    """The error of whatever block_tables_fork or block_tables_compact found wrong with its tensors."""
    for name, t in required.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    _refuse(what, here, **{name: (t, _I32) for name, t in (*required.items(), *optional.items())}, workspace=(workspace, None))
    table = required["block_table"].shape
    if len(table) != 2:
        raise ValueError(f"{what}: block_table must be [B][MBS]")
    raise ValueError(f"{what}: shapes do not match (block_table, block_table_out [B][MBS]; context_lens, context_lens_out, parents "
                     "[B]; refs, free_list, held [NB]; free_count, pair_count [1]; pairs [B][2], to compact [NB // 2][2])")


def block_tables_fork(block_table, context_lens, parents, block_table_out, context_lens_out, refs, free_list, free_count,
                      pairs, pair_count, bs, held=None, workspace=None, stream=None) -> None:
    """Row b takes the sequence of row parents[b] (int32 [B], -1: none; None: every row its own), sharing
    its blocks but for a partly filled last one; references counted anew, blocks without any free
    (see pkv.h).  refs, free_list int32 [NB], free_count, pair_count int32 [1], pairs int32 [B][2]:
    the copies to run with kv_block_copy(..., pairs, count=pair_count).  held: int32 [NB] or None."""
    here = _current_device()
    ints = (block_table, context_lens, block_table_out, context_lens_out, refs, free_list, free_count, pairs, pair_count)
    try:
        ok = _ready(here, (*ints, parents, held, workspace)) and all([t.dtype is _I32 for t in ints]) and \
            (parents is None or parents.dtype is _I32) and (held is None or held.dtype is _I32)
        (B, MBS), NB = block_table.shape, free_list.numel()
        ok = ok and block_table_out.numel() == B * MBS and context_lens.numel() == B and context_lens_out.numel() == B and \
            refs.numel() == NB and free_count.numel() == 1 and pair_count.numel() == 1 and pairs.numel() == 2 * B and \
            (parents is None or parents.numel() == B) and (held is None or held.numel() == NB)
    except (AttributeError, ValueError):   # not a tensor, or not a table
        ok = False
    if not ok:
        _share_refuse("block_tables_fork", here, workspace, dict(parents=parents, held=held), block_table=block_table,
                      context_lens=context_lens, block_table_out=block_table_out, context_lens_out=context_lens_out, refs=refs,
                      free_list=free_list, free_count=free_count, pairs=pairs, pair_count=pair_count)
    status = lib().pkv_block_tables_fork(
        block_table.data_ptr(), context_lens.data_ptr(), _ptr(parents), _ptr(held), block_table_out.data_ptr(),
        context_lens_out.data_ptr(), refs.data_ptr(), free_list.data_ptr(), free_count.data_ptr(), pairs.data_ptr(),
        pair_count.data_ptr(), B, MBS, int(bs), NB, _ptr(workspace), _bytes(workspace), _stream(stream, here))
    if status:
        _check(status)


def block_tables_compact(block_table, context_lens, block_table_out, refs, free_list, free_count, pairs, pair_count, bs,
                         held=None, workspace=None, stream=None) -> None:
    """The blocks in use moved to the lowest ids (see pkv.h); pairs int32 [NB // 2][2], the other
    tensors as block_tables_fork."""
    here = _current_device()
    ints = (block_table, context_lens, block_table_out, refs, free_list, free_count, pairs, pair_count)
    try:
        ok = _ready(here, (*ints, held, workspace)) and all([t.dtype is _I32 for t in ints]) and (held is None or held.dtype is _I32)
        (B, MBS), NB = block_table.shape, free_list.numel()
        ok = ok and block_table_out.numel() == B * MBS and context_lens.numel() == B and refs.numel() == NB and \
            free_count.numel() == 1 and pair_count.numel() == 1 and pairs.numel() == NB // 2 * 2 and (held is None or held.numel() == NB)
    except (AttributeError, ValueError):   # not a tensor, or not a table
        ok = False
    if not ok:
        _share_refuse("block_tables_compact", here, workspace, dict(held=held), block_table=block_table, context_lens=context_lens,
                      block_table_out=block_table_out, refs=refs, free_list=free_list, free_count=free_count, pairs=pairs,
                      pair_count=pair_count)
    status = lib().pkv_block_tables_compact(
        block_table.data_ptr(), context_lens.data_ptr(), _ptr(held), block_table_out.data_ptr(), refs.data_ptr(),
        free_list.data_ptr(), free_count.data_ptr(), pairs.data_ptr(), pair_count.data_ptr(), B, MBS, int(bs), NB,
        _ptr(workspace), _bytes(workspace), _stream(stream, here))
    if status:
        _check(status)


# ------------------------------------------------------------- rotary positions

_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


def rope_turns(rot, base=10000.0, scaling="none", factor=1.0, original=1, low=1.0, high=32.0, device="cuda") -> torch.Tensor:
    """The angles per position of rot // 2 dimension pairs, as fractions of a turn in 2^-64 units (int64
    [rot // 2], the bits of uint64): the `turns` of rope and rope_append, made once.  scaling: "none",
    "linear", "base" or "parts", for contexts `factor` times `original` tokens (see pkv.h)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"rope_turns: scaling {scaling!r} (one of {', '.join(_SCALINGS)})")
    turns = torch.zeros(max(1, int(rot) // 2), dtype=_I64)
    _check(lib().pkv_rope_turns(turns.data_ptr(), int(rot), float(base), _SCALINGS[scaling], float(factor), float(original),
                                float(low), float(high)))
    return turns.to(device)


def _heads(what, name, t, T, H, d) -> int:
    """Elements between the tokens of t [T][H][d], whose rows [H][d] are contiguous."""
    token, head, one = t.stride()
    if (one != 1 and d > 1) or (head != d and H > 1):
        raise ValueError(f"{what}: the heads of a token of {name} must be contiguous")
    return token if T > 1 else H * d


def _rope_check(what, q_out, q, positions, turns, here, **more):
    for name, (t, dtype, strided) in {"q_out": (q_out, None, False), "q": (q, None, True), "positions": (positions, _I32, False),
                                      "turns": (turns, _I64, False), **more}.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
        if t.get_device() != here:   # the kernels run on the current device
            raise ValueError(f"{what}: {name} is on device {t.get_device()}, the current one is {here}")
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not strided and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dim() != 3 or q_out.shape != q.shape or positions.numel() != q.shape[0]:
        raise ValueError(f"{what}: shapes do not match [T][Hq][d] / [T]")


def rope_append(q_out, q, k_new, v_new, k_cache, v_cache, positions, slot_mapping, turns, interleaved=False, mscale=1.0,
                stream=None) -> None:
    """q [T][Hq][d] rotated by positions[t] (int32) into q_out (fp32 or bf16); k_new [T][Hkv][d] rotated
    and v_new as it is into cache slots slot_mapping[t] (int64, < 0: none).  The tokens of q, k_new and
    v_new may be any distance apart (views of packed rows).  turns: rope_turns(rot), of the first rot
    dimensions; pairs (j, j + rot / 2), or (2j, 2j + 1) when interleaved."""
    what, here = "rope_append", _current_device()
    try:   # the common outcome of the checks below, without their detours
        dt, shape = q.dtype, q.shape
        ok = (_ready(here, (q_out, k_cache, v_cache, positions, slot_mapping, turns)) and q.get_device() == here and
              k_new.get_device() == here and v_new.get_device() == here and k_new.dtype is dt and v_new.dtype is dt and
              k_cache.dtype is dt and v_cache.dtype is dt and positions.dtype is _I32 and slot_mapping.dtype is _I64 and
              turns.dtype is _I64 and len(shape) == 3 and q_out.shape == shape and positions.numel() == shape[0])
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        dt = getattr(q, "dtype", None)
        _rope_check(what, q_out, q, positions, turns, here, k_new=(k_new, dt, True), v_new=(v_new, dt, True),
                    k_cache=(k_cache, dt, False), v_cache=(v_cache, dt, False), slot_mapping=(slot_mapping, _I64, False))
        shape = q.shape
    T, Hq, d = shape
    cache, new = k_cache.shape, k_new.shape
    if len(cache) != 4 or v_cache.shape != cache or cache[3] != d or slot_mapping.numel() != T or len(new) != 3 or \
            v_new.shape != new or new[0] != T or new[1] != cache[1] or new[2] != d:
        raise ValueError("rope_append: shapes do not match (k_new, v_new [T][Hkv][d], caches [NB][Hkv][bs][d], slot_mapping [T])")
    NB, Hkv, bs, _ = cache
    status = lib().pkv_rope_append(
        q_out.data_ptr(), _dtype(q_out), q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), _dtype(k_cache), _heads(what, "q", q, T, Hq, d),
        _heads(what, "k_new", k_new, T, Hkv, d), _heads(what, "v_new", v_new, T, Hkv, d), positions.data_ptr(), turns.data_ptr(),
        2 * turns.numel(), 1 if interleaved else 0, float(mscale), k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), T, Hq,
        Hkv, d, bs, NB, _stream(stream, here))
    if status:
        _check(status)


def rope(q_out, q, k_out, k, positions, turns, interleaved=False, mscale=1.0, inverse=False, stream=None) -> None:
    """q [T][Hq][d] rotated into q_out (fp32 or bf16) and k [T][Hkv][d] into k_out (its type; both None:
    q alone), as rope_append does.  inverse: rotated back (the gradient of the rotation)."""
    what, here = "rope", _current_device()
    with_k = k is not None or k_out is not None
    try:
        dt, shape = q.dtype, q.shape
        ok = (_ready(here, (q_out, positions, turns, k_out)) and q.get_device() == here and positions.dtype is _I32 and
              turns.dtype is _I64 and len(shape) == 3 and q_out.shape == shape and positions.numel() == shape[0] and
              (not with_k or (k.get_device() == here and k.dtype is dt and k_out.dtype is dt)))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        dt = getattr(q, "dtype", None)
        _rope_check(what, q_out, q, positions, turns, here, **({"k": (k, dt, True), "k_out": (k_out, dt, False)} if with_k else {}))
        shape = q.shape
    T, Hq, d = shape
    Hkv, k_stride = 1, 0
    if with_k:
        rows = k.shape
        if len(rows) != 3 or k_out.shape != rows or rows[0] != T or rows[2] != d:
            raise ValueError("rope: k and k_out must be [T][Hkv][d]")
        Hkv = rows[1]
        k_stride = _heads(what, "k", k, T, Hkv, d)
    status = lib().pkv_rope(
        q_out.data_ptr(), _dtype(q_out), _ptr(k_out), q.data_ptr(), _ptr(k), _dtype(q), _heads(what, "q", q, T, Hq, d), k_stride,
        positions.data_ptr(), turns.data_ptr(), 2 * turns.numel(), 1 if interleaved else 0, float(mscale), 1 if inverse else 0, T, Hq, Hkv,
        d, _stream(stream, here))
    if status:
        _check(status)


# --------------------------------------------------------------- drafted tokens

def verify_drafts(accepted, tokens, target_probs, draft_tokens, cu_drafts, uniforms, draft_probs=None, context_lens=None,
                  context_lens_out=None, stream=None) -> None:
    """Drafts accepted against the target's probabilities, and a next token for every sequence (see pkv.h).

    accepted int32 [B]; tokens int32 [D + B]; target_probs [D + B][V] and draft_probs [D][V] (or None: the
    drafts were chosen, not drawn), fp32 or bf16, rows any distance apart; draft_tokens int32 [D];
    cu_drafts int32 [B + 1]; uniforms fp32 [D + B]; context_lens, context_lens_out int32 [B]: the
    lengths with the drafts, and without the rejected ones (may be the same)."""
    what, here = "verify_drafts", _current_device()
    ints = (accepted, tokens, draft_tokens, cu_drafts)
    try:
        dt = target_probs.dtype
        ok = (_ready(here, (*ints, uniforms, context_lens, context_lens_out)) and accepted.dtype is _I32 and tokens.dtype is _I32 and
              draft_tokens.dtype is _I32 and cu_drafts.dtype is _I32 and uniforms.dtype is _F32 and
              (context_lens is None or context_lens.dtype is _I32) and (context_lens_out is None or context_lens_out.dtype is _I32) and
              target_probs.get_device() == here and (draft_probs is None or (draft_probs.get_device() == here and draft_probs.dtype is dt)))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(what, here, accepted=(accepted, _I32), tokens=(tokens, _I32), draft_tokens=(draft_tokens, _I32),
                cu_drafts=(cu_drafts, _I32), uniforms=(uniforms, _F32), context_lens_out=(context_lens_out, _I32))
        if context_lens is not None:
            _refuse(what, here, context_lens=(context_lens, _I32))
        for name, t in (("target_probs", target_probs), ("draft_probs", draft_probs)):
            if t is None and name == "draft_probs":
                continue
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.get_device() != here:
                raise ValueError(f"{what}: {name} is on {t.device}, the current device is {here}")
            if t.dtype is not target_probs.dtype:
                raise TypeError(f"{name} must be {target_probs.dtype}, got {t.dtype}")
    rows = target_probs.shape
    B, D = accepted.numel(), draft_tokens.numel()
    if len(rows) != 2 or rows[0] != D + B or tokens.numel() != D + B or uniforms.numel() != D + B or cu_drafts.numel() != B + 1 or \
            (draft_probs is not None and (draft_probs.dim() != 2 or draft_probs.shape[0] != D or draft_probs.shape[1] != rows[1])) or \
            (context_lens is not None and context_lens.numel() != B) or \
            (context_lens_out is not None and context_lens_out.numel() != B):
        raise ValueError("verify_drafts: shapes do not match")
    V = rows[1]

    def apart(name, t, n):   # elements between rows
        row, one = t.stride()
        if one != 1 and V > 1:
            raise ValueError(f"verify_drafts: {name} must be rows of contiguous probabilities")
        return row if n > 1 else V

    target_apart = apart("target_probs", target_probs, D + B)
    draft_apart = apart("draft_probs", draft_probs, D) if draft_probs is not None else 0
    status = lib().pkv_verify_drafts(
        accepted.data_ptr(), tokens.data_ptr(), target_probs.data_ptr(), _ptr(draft_probs) if D > 0 else 0, _dtype(target_probs),
        target_apart, draft_apart, draft_tokens.data_ptr(), cu_drafts.data_ptr(), uniforms.data_ptr(),
        _ptr(context_lens), _ptr(context_lens_out), B, D, V, _stream(stream, here))
    if status:
        _check(status)


# ----------------------------------------------------- windows with first tokens

def paged_attention_sinks_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, bs, MBS, window, sinks, num_splits=0) -> int:
    return int(lib().pkv_paged_attention_sinks_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, bs, MBS, window, sinks, num_splits))


def paged_attention_sinks(out, q, k_cache, v_cache, block_table, context_lens, scale, window, sinks, cu_q=None, max_q=1,
                          lse=None, num_splits=0, workspace=None, stream=None) -> None:
    """paged_attention with a sliding window whose first `sinks` tokens stay visible: the row at position p
    sees the keys t <= p with t < sinks or t > p - window.

    q, out [Tq][Hq][d] fp32; cu_q int32 [B+1] (None: one query per sequence)."""
    what, here = "paged_attention_sinks", _current_device()
    try:
        ok = (_ready(here, (out, q, k_cache, v_cache, block_table, context_lens, lse, cu_q, workspace)) and q.dtype is _F32 and
              out.dtype is _F32 and v_cache.dtype is k_cache.dtype and block_table.dtype is _I32 and context_lens.dtype is _I32 and
              (lse is None or lse.dtype is _F32) and (cu_q is None or cu_q.dtype is _I32))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(what, here, q=(q, _F32), out=(out, _F32), k_cache=(k_cache, None),
                v_cache=(v_cache, getattr(k_cache, "dtype", None)), block_table=(block_table, _I32),
                context_lens=(context_lens, _I32), lse=(lse, _F32), cu_q=(cu_q, _I32), workspace=(workspace, None))
    dt, rows, cache, table, B = _dtype(k_cache), q.shape, k_cache.shape, block_table.shape, context_lens.numel()
    if len(rows) != 3 or len(cache) != 4:
        raise ValueError(f"{what}: q must be [rows][Hq][d] and the caches [NB][Hkv][bs][d]")
    NB, Hkv, bs, d = cache
    Tq, Hq, dq = rows
    if dq != d or out.shape != rows or v_cache.shape != cache or len(table) != 2 or table[0] != B or \
            (cu_q.numel() != B + 1 if cu_q is not None else Tq != B) or (lse is not None and lse.numel() != Tq * Hq):
        raise ValueError(f"{what}: shapes do not match")
    status = lib().pkv_paged_attention_sinks(
        out.data_ptr(), _ptr(lse), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), dt, block_table.data_ptr(),
        context_lens.data_ptr(), _ptr(cu_q), B, Tq, int(max_q), Hq, Hkv, d, bs, table[1], NB, float(scale), int(window), int(sinks),
        int(num_splits), _ptr(workspace), _bytes(workspace), _stream(stream, here))
    if status:
        _check(status)
