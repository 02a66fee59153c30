"""Paged FP8-KV decode attention for NVIDIA B200 (sm_100a).

A thin Python binding over the C-ABI library ``libpagedkv.so`` (declared in
``include/pagedkv.h``).  Each function here only checks and marshals its torch
tensors into pointers and sizes and calls the C entry point of the same name
on the current CUDA stream; every step of the computation runs in the
library's CUDA kernels.  Nothing here falls back to PyTorch or to the CPU: if
the library is missing or fails, the call raises.

Tensors (all on one CUDA device, contiguous):
  q            [B][Hq][D]      torch.bfloat16
  k/v caches   [NP][Hkv][P][D] torch.uint8 (E4M3 codes) or torch.bfloat16
  k_new/v_new  [B][Hkv][D]     torch.bfloat16
  page_table   [B][MP]         torch.int32
  seq_lens     [B]             torch.int32   (counts the new token)
  page_tags    [NP]            torch.int32 / uint32 view (raw 32-bit tags)
  expected     [B][MP]         same dtype as page_tags
  abort        [B]             torch.uint8

INT4 caches are pairs of tensors, K and V each:
  codes        [NP][Hkv][P][D/2]      torch.uint8 (two 4-bit codes per byte)
  params       [NP][Hkv][P][D/64][2]  torch.bfloat16 (scale, minimum of 64 dims)

Page tables and slots (kv_extend_tables, kv_write_slots_*, kv_read_slots_*):
  old/new_lens [B]             torch.int32
  free_pages   [<= NP]         torch.int32   (a stack; top at num_free - 1)
  num_free     [1]             torch.int32
  slot_map     [T]             torch.int32   (page * P + offset, or -1)
  cu_tokens    [B + 1]         torch.int32
  failed       [B]             torch.uint8
  token rows   [T][Hkv][D]     torch.bfloat16 (rows may be part of wider ones)

INT4 weight dequantisation GEMV (int4_dequant_gemv):
  x            [B][k]                      torch.bfloat16
  w_tiles      [n/128][k/256][128][128]    torch.uint8 (two signed 4-bit codes per byte)
  scales       [n/128][k/group][128]       torch.bfloat16
  y            [B][n]                      torch.bfloat16
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedkv.so")

PKV_OK = 0
PKV_KV_FP8 = 0
PKV_KV_BF16 = 1
PKV_KV_INT4 = 2
INT4_GROUP = 64   # dims that share a (scale, minimum) pair of an INT4 cache
_STATUS = {1: "invalid argument", 2: "workspace", 3: "unsupported", 4: "CUDA error"}


class PagedKVError(RuntimeError):
    """A library call returned a non-OK status."""

    def __init__(self, func: str, status: int, message: str):
        super().__init__(f"{func}: {_STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m paged_fp8_kv_attn_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        i64 = ctypes.c_int64
        attn = [P, i32, P, i32, i32, i32, i32, i32, i32, f32]   # page_table .. sm_scale
        attn_out = [P, P, P, P, sz, i32, P]                     # abort .. stream
        slots = [P, i32, i32, i32, i32]                         # slot_map .. page_size
        sig = {
            "kv_tag_check": [P, i32, P, P, i32, P, i32, i32, P, P, P],
            "kv_append_fp8": [P, P, P, i32, P, i32, i32, i32, i32, f32, f32, P, P, i32, P, P],
            "kv_append_bf16": [P, P, P, i32, P, i32, i32, i32, i32, P, P, i32, P, P],
            "kv_requant_pages_fp8": [P, i32, P, P, i32, P, i32, i32, i32, i32, f32, P],
            "kv_retag_pages": [P, i32, P, i32, P],
            "kv_expected_tags": [P, i32, P, i32, P, i32, i32, P, P],
            "kv_check_append_fp8": [P, i32, P, P, i32, P, i32, i32, P, P, i32, i32, f32, f32, P, P,
                                    P, P, P],
            "kv_check_append_bf16": [P, i32, P, P, i32, P, i32, i32, P, P, i32, i32, P, P, P, P,
                                     P],
            "paged_decode_attn_fp8": [P, P, P, f32, f32, P, i32, P, i32, i32, i32, i32, i32, i32,
                                      f32, P, P, P, P, sz, i32, P],
            "paged_decode_attn_bf16": [P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, f32, P,
                                       P, P, P, sz, i32, P],
            "paged_decode_attn_fp8_prefix": [P, P, P, f32, f32, P, i32, P, i32, i32, i32, i32, i32,
                                             i32, f32, P, P, P, P, sz, i32, P, P],
            "kv_tag_check_window": [P, i32, P, P, i32, P, i32, i32, i32, i32, P, P, P],
            "kv_append_int4": [P, P, P, i32, P, i32, i32, i32, i32, P, P, P, P, i32, P, P],
            "kv_check_append_int4": [P, i32, P, P, i32, P, i32, i32, P, P, i32, i32, P, P, P, P, P,
                                     P, P],
            "kv_requant_pages_int4": [P, i32, P, P, P, i32, P, i32, i32, i32, i32, P],
            "kv_write_slots_fp8": [P, P, i64, i64, *slots, f32, f32, P, P, i32, P],
            "kv_write_slots_bf16": [P, P, i64, i64, *slots, P, P, i32, P],
            "kv_write_slots_int4": [P, P, i64, i64, *slots, P, P, P, P, i32, P],
            "kv_read_slots_fp8": [*slots, f32, f32, P, P, i32, P, P, i64, i64, P],
            "kv_read_slots_bf16": [*slots, P, P, i32, P, P, i64, i64, P],
            "kv_read_slots_int4": [*slots, P, P, P, P, i32, P, P, i64, i64, P],
            "kv_extend_tables": [P, P, i32, i32, P, i32, P, P, i32, P, i32, P, P, P, i32, P, P, P],
            "paged_decode_attn_int4": [P, P, P, P, P, *attn, *attn_out],
            "paged_decode_attn_fp8_window": [P, P, P, f32, f32, *attn, i32, i32, *attn_out],
            "paged_decode_attn_bf16_window": [P, P, P, *attn, i32, i32, *attn_out],
            "paged_decode_attn_int4_window": [P, P, P, P, P, *attn, i32, i32, *attn_out],
            "int4_dequant_gemv": [P, P, P, i32, i32, i32, i32, P, P, P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = i32
        lib.paged_decode_attn_fp8_noalloc.argtypes = [P, P, P, f32, f32, P, i32, P, i32, i32,
                                                      i32, i32, i32, i32, f32, P, P, P, i32, P]
        lib.paged_decode_attn_fp8_noalloc.restype = i32
        lib.paged_decode_attn_fp8_noalloc_scratch_bytes.argtypes = []
        lib.paged_decode_attn_fp8_noalloc_scratch_bytes.restype = sz
        lib.paged_decode_attn_fp8_noalloc_status.argtypes = [P, P]
        lib.paged_decode_attn_fp8_noalloc_status.restype = i32
        pi32 = ctypes.POINTER(i32)
        lib.paged_decode_attn_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, pi32,
                                               pi32, pi32]
        lib.paged_decode_attn_plan.restype = i32
        lib.paged_decode_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.paged_decode_attn_workspace_size.restype = sz
        lib.paged_decode_attn_fp8_prefix_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.paged_decode_attn_fp8_prefix_workspace_size.restype = sz
        lib.pkv_last_error.argtypes = []
        lib.pkv_last_error.restype = ctypes.c_char_p
        lib.pkv_version.argtypes = []
        lib.pkv_version.restype = i32
        _lib = lib
    return _lib


def library() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    return _load()


def _check(name: str, status: int):
    if status != PKV_OK:
        raise PagedKVError(name, status, _load().pkv_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


# (the handle alone: torch.cuda.current_stream() builds an object, 3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream=None):
    return _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _need(t, dtype, ndim, name):
    # (one line of cheap tests for the usual case: a call's host time is mostly these)
    if t is not None and t.is_cuda and t.dim() == ndim and t.is_contiguous() and (
            t.dtype is dtype or type(dtype) is tuple and t.dtype in dtype):
        return t
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _on(stream):
    """Device index and stream handle of a call."""
    if stream is None:
        dev = torch.cuda.current_device()
        return dev, _raw_stream(dev)
    return stream.device_index, stream.cuda_stream


def _args(dev, anchors, *specs):
    """Each (name, tensor, dtype, shape): contiguous, on the call's device; anchors, the
    tensors that gave the shapes and are checked otherwise: on the call's device."""
    for t in anchors:
        if t.get_device() != dev:
            raise ValueError(f"tensors must be on the call's device {dev}, got {t.device}")
    for name, t, dtype, shape in specs:
        if t is None or t.get_device() != dev or t.dtype is not dtype or t.shape != shape \
                or not t.is_contiguous():
            _need(t, dtype, len(shape), name)
            _match(name, t, shape)
            raise ValueError(f"{name} must be on the call's device {dev}, got {t.device}")


def _match(name, t, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _i32(value, name):
    """An int argument of the C call (ctypes would drop its bits past 32)."""
    value = int(value)
    if not -2**31 <= value < 2**31:
        raise ValueError(f"{name} must fit in 32 bits, got {value}")
    return value


def _window(window, sinks):
    """(window, sinks) of the C call: 2^31 - 1 stands for anything larger, since no
    length passes it, and -1 for anything negative, which the call refuses."""
    return tuple(min(max(int(x), -1), 2**31 - 1) for x in (window, sinks))


def _tag_dtype(t, name):
    """The dtype of tags: one of _TAG_DTYPES."""
    return _need(t, _TAG_DTYPES, 1, name).dtype


def _int4_shape(k_codes):
    """(NP, Hkv, P, D) of an INT4 cache with these K codes."""
    NP, Hkv, P, half = _need(k_codes, torch.uint8, 4, "k_codes").shape
    return NP, Hkv, P, 2 * half


def _int4_specs(shape, k_params, v_codes, v_params):
    """Of the tensors that go with the K codes."""
    NP, Hkv, P, D = shape
    codes, params = (NP, Hkv, P, D // 2), (NP, Hkv, P, D // INT4_GROUP, 2)
    return (("k_params", k_params, torch.bfloat16, params), ("v_codes", v_codes, torch.uint8, codes),
            ("v_params", v_params, torch.bfloat16, params))


_TAG_DTYPES = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)


def kv_tag_check(page_tags, page_table, expected_tags, seq_lens, page_size, abort_out,
                 num_aborted=None, stream=None):
    """Batched page-tag integrity check; writes abort_out [B] (uint8)."""
    _need(page_tags, _TAG_DTYPES, 1, "page_tags")
    _need(page_table, torch.int32, 2, "page_table")
    _need(expected_tags, _TAG_DTYPES, 2, "expected_tags")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(abort_out, torch.uint8, 1, "abort_out")
    B, MP = page_table.shape
    if num_aborted is not None:
        _need(num_aborted, torch.int32, 1, "num_aborted")
    _check("kv_tag_check", _load().kv_tag_check(
        _ptr(page_tags), page_tags.shape[0], _ptr(page_table), _ptr(expected_tags), MP,
        _ptr(seq_lens), B, page_size, _ptr(abort_out), _ptr(num_aborted), _stream(stream)))


def kv_tag_check_window(page_tags, page_table, expected_tags, seq_lens, page_size, window, sinks,
                        abort_out, num_aborted=None, stream=None):
    """kv_tag_check of the pages that hold one of the last `window` or the first
    `sinks` tokens of a request; entries of hidden pages are not read."""
    i32 = torch.int32
    B, MP = _need(page_table, i32, 2, "page_table").shape
    tag = _tag_dtype(page_tags, "page_tags")
    dev, handle = _on(stream)
    _args(dev, (page_tags, page_table), ("expected_tags", expected_tags, tag, (B, MP)), ("seq_lens", seq_lens, i32, (B,)),
          ("abort_out", abort_out, torch.uint8, (B,)))
    if num_aborted is not None:
        _args(dev, (), ("num_aborted", num_aborted, i32, (1,)))
    _check("kv_tag_check_window", _load().kv_tag_check_window(
        _ptr(page_tags), page_tags.shape[0], _ptr(page_table), _ptr(expected_tags), MP,
        _ptr(seq_lens), B, _i32(page_size, "page_size"), *_window(window, sinks), _ptr(abort_out),
        _ptr(num_aborted), handle))


def kv_retag_pages(page_tags, pages, stream=None):
    """Bump (mod 2^32) the tag of every listed page id inside the pool, in place."""
    _need(page_tags, _TAG_DTYPES, 1, "page_tags")
    _need(pages, torch.int32, 1, "pages")
    _check("kv_retag_pages", _load().kv_retag_pages(
        _ptr(page_tags), page_tags.shape[0], _ptr(pages), pages.shape[0], _stream(stream)))


def kv_expected_tags(page_tags, page_table, seq_lens, page_size, expected_tags, stream=None):
    """Rebuild each request's expected tags from the current page tags, in place."""
    _need(page_tags, _TAG_DTYPES, 1, "page_tags")
    _need(page_table, torch.int32, 2, "page_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(expected_tags, _TAG_DTYPES, 2, "expected_tags")
    B, MP = page_table.shape
    _check("kv_expected_tags", _load().kv_expected_tags(
        _ptr(page_tags), page_tags.shape[0], _ptr(page_table), MP, _ptr(seq_lens), B, page_size,
        _ptr(expected_tags), _stream(stream)))


def kv_append_fp8(k_new, v_new, page_table, seq_lens, page_size, k_scale, v_scale,
                  k_cache, v_cache, abort=None, stream=None):
    """Quantise each request's new K/V token to E4M3 and write it into its page."""
    _need(k_new, torch.bfloat16, 3, "k_new")
    _need(v_new, torch.bfloat16, 3, "v_new")
    _need(page_table, torch.int32, 2, "page_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(k_cache, torch.uint8, 4, "k_cache")
    _need(v_cache, torch.uint8, 4, "v_cache")
    if abort is not None:
        _need(abort, torch.uint8, 1, "abort")
    B, Hkv, D = k_new.shape
    _check("kv_append_fp8", _load().kv_append_fp8(
        _ptr(k_new), _ptr(v_new), _ptr(page_table), page_table.shape[1], _ptr(seq_lens), B, Hkv,
        D, page_size, float(k_scale), float(v_scale), _ptr(k_cache), _ptr(v_cache),
        k_cache.shape[0], _ptr(abort), _stream(stream)))


def kv_append_bf16(k_new, v_new, page_table, seq_lens, page_size, k_cache, v_cache,
                   abort=None, stream=None):
    """Write each request's new BF16 K/V token into its page."""
    _need(k_new, torch.bfloat16, 3, "k_new")
    _need(v_new, torch.bfloat16, 3, "v_new")
    _need(page_table, torch.int32, 2, "page_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    if abort is not None:
        _need(abort, torch.uint8, 1, "abort")
    B, Hkv, D = k_new.shape
    _check("kv_append_bf16", _load().kv_append_bf16(
        _ptr(k_new), _ptr(v_new), _ptr(page_table), page_table.shape[1], _ptr(seq_lens), B, Hkv,
        D, page_size, _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(abort),
        _stream(stream)))


def kv_check_append_fp8(page_tags, page_table, expected_tags, seq_lens, page_size, k_new, v_new,
                        k_scale, v_scale, k_cache, v_cache, abort_out, num_aborted=None,
                        stream=None):
    """kv_tag_check then kv_append_fp8 (with that abort mask) in one kernel."""
    _need(page_tags, _TAG_DTYPES, 1, "page_tags")
    _need(page_table, torch.int32, 2, "page_table")
    _need(expected_tags, _TAG_DTYPES, 2, "expected_tags")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(k_new, torch.bfloat16, 3, "k_new")
    _need(v_new, torch.bfloat16, 3, "v_new")
    _need(k_cache, torch.uint8, 4, "k_cache")
    _need(v_cache, torch.uint8, 4, "v_cache")
    _need(abort_out, torch.uint8, 1, "abort_out")
    if num_aborted is not None:
        _need(num_aborted, torch.int32, 1, "num_aborted")
    B, MP = page_table.shape
    _, Hkv, D = k_new.shape
    _check("kv_check_append_fp8", _load().kv_check_append_fp8(
        _ptr(page_tags), k_cache.shape[0], _ptr(page_table), _ptr(expected_tags), MP,
        _ptr(seq_lens), B, page_size, _ptr(k_new), _ptr(v_new), Hkv, D, float(k_scale),
        float(v_scale), _ptr(k_cache), _ptr(v_cache), _ptr(abort_out), _ptr(num_aborted),
        _stream(stream)))


def kv_check_append_bf16(page_tags, page_table, expected_tags, seq_lens, page_size, k_new, v_new,
                         k_cache, v_cache, abort_out, num_aborted=None, stream=None):
    """kv_tag_check then kv_append_bf16 (with that abort mask) in one kernel."""
    _need(page_tags, _TAG_DTYPES, 1, "page_tags")
    _need(page_table, torch.int32, 2, "page_table")
    _need(expected_tags, _TAG_DTYPES, 2, "expected_tags")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(k_new, torch.bfloat16, 3, "k_new")
    _need(v_new, torch.bfloat16, 3, "v_new")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    _need(abort_out, torch.uint8, 1, "abort_out")
    if num_aborted is not None:
        _need(num_aborted, torch.int32, 1, "num_aborted")
    B, MP = page_table.shape
    _, Hkv, D = k_new.shape
    _check("kv_check_append_bf16", _load().kv_check_append_bf16(
        _ptr(page_tags), k_cache.shape[0], _ptr(page_table), _ptr(expected_tags), MP,
        _ptr(seq_lens), B, page_size, _ptr(k_new), _ptr(v_new), Hkv, D, _ptr(k_cache),
        _ptr(v_cache), _ptr(abort_out), _ptr(num_aborted), _stream(stream)))


def kv_append_int4(k_new, v_new, page_table, seq_lens, page_size, k_codes, k_params, v_codes,
                   v_params, abort=None, stream=None):
    """Quantise each request's new K/V token to 4 bits and write it into its page."""
    shape = NP, Hkv, P, D = _int4_shape(k_codes)
    B, MP = _need(page_table, torch.int32, 2, "page_table").shape
    dev, handle = _on(stream)
    _args(dev, (k_codes, page_table), *_int4_specs(shape, k_params, v_codes, v_params),
          *_append_specs(k_new, v_new, seq_lens, page_size, shape, B))
    if abort is not None:
        _args(dev, (), ("abort", abort, torch.uint8, (B,)))
    _check("kv_append_int4", _load().kv_append_int4(
        _ptr(k_new), _ptr(v_new), _ptr(page_table), MP, _ptr(seq_lens), B, Hkv, D, P,
        _ptr(k_codes), _ptr(k_params), _ptr(v_codes), _ptr(v_params), NP, _ptr(abort), handle))


def kv_check_append_int4(page_tags, page_table, expected_tags, seq_lens, page_size, k_new, v_new,
                         k_codes, k_params, v_codes, v_params, abort_out, num_aborted=None,
                         stream=None):
    """kv_tag_check then kv_append_int4 (with that abort mask) in one kernel."""
    shape = NP, Hkv, P, D = _int4_shape(k_codes)
    B, MP = _need(page_table, torch.int32, 2, "page_table").shape
    tag = _tag_dtype(page_tags, "page_tags")
    dev, handle = _on(stream)
    _args(dev, (k_codes, page_table), *_int4_specs(shape, k_params, v_codes, v_params),
          *_append_specs(k_new, v_new, seq_lens, page_size, shape, B),
          ("page_tags", page_tags, tag, (NP,)), ("expected_tags", expected_tags, tag, (B, MP)),
          ("abort_out", abort_out, torch.uint8, (B,)))
    if num_aborted is not None:
        _args(dev, (), ("num_aborted", num_aborted, torch.int32, (1,)))
    _check("kv_check_append_int4", _load().kv_check_append_int4(
        _ptr(page_tags), NP, _ptr(page_table), _ptr(expected_tags), MP, _ptr(seq_lens), B, P,
        _ptr(k_new), _ptr(v_new), Hkv, D, _ptr(k_codes), _ptr(k_params), _ptr(v_codes),
        _ptr(v_params), _ptr(abort_out), _ptr(num_aborted), handle))


def _append_specs(k_new, v_new, seq_lens, page_size, shape, B):
    """Of an append to a cache of that shape."""
    _, Hkv, P, D = shape
    if page_size != P:
        raise ValueError(f"page_size is {page_size}, the cache's pages hold {P} tokens")
    new = (B, Hkv, D)
    return (("k_new", k_new, torch.bfloat16, new), ("v_new", v_new, torch.bfloat16, new),
            ("seq_lens", seq_lens, torch.int32, (B,)))


def _token_rows(t, name, T, Hkv, D, dev):
    """Row stride of [T][Hkv][D] token rows, each row contiguous."""
    if t is None or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    _match(name, t, (T, Hkv, D))
    row = Hkv * D
    if T < 2 and t.is_contiguous():
        return row
    stride = t.stride()
    if T and (stride[2] != 1 or (Hkv > 1 and stride[1] != D) or (T > 1 and stride[0] < row)):
        raise ValueError(f"{name} must hold each token's [Hkv][D] values contiguously")
    return stride[0] if T > 1 else row


def _slot_call(name, slot_map, pools, scales, k, v, shape, specs, write, stream):
    T = _need(slot_map, torch.int32, 1, "slot_map").numel()
    NP, Hkv, P, D = shape
    dev, handle = _on(stream)
    _args(dev, (slot_map, pools[0]), *specs)
    ks, vs = _token_rows(k, "k", T, Hkv, D, dev), _token_rows(v, "v", T, Hkv, D, dev)
    rows = (k.data_ptr(), v.data_ptr(), ks, vs)
    cache = (slot_map.data_ptr(), T, Hkv, D, P, *scales, *[t.data_ptr() for t in pools], NP)
    fn = getattr(_load(), name)
    _check(name, fn(*rows, *cache, handle) if write else fn(*cache, *rows, handle))


def kv_write_slots_fp8(k_new, v_new, slot_map, k_scale, v_scale, k_cache, v_cache, stream=None):
    """Quantise token rows to E4M3 and write row i into slot slot_map[i] (negative: skipped)."""
    shape = _need(k_cache, torch.uint8, 4, "k_cache").shape
    _slot_call("kv_write_slots_fp8", slot_map, (k_cache, v_cache), (float(k_scale), float(v_scale)),
               k_new, v_new, shape, (("v_cache", v_cache, torch.uint8, shape),), True, stream)


def kv_write_slots_bf16(k_new, v_new, slot_map, k_cache, v_cache, stream=None):
    """Write token row i into slot slot_map[i] of a BF16 cache (negative: skipped)."""
    shape = _need(k_cache, torch.bfloat16, 4, "k_cache").shape
    _slot_call("kv_write_slots_bf16", slot_map, (k_cache, v_cache), (), k_new, v_new, shape,
               (("v_cache", v_cache, torch.bfloat16, shape),), True, stream)


def kv_write_slots_int4(k_new, v_new, slot_map, k_codes, k_params, v_codes, v_params, stream=None):
    """Quantise token rows to 4 bits and write row i into slot slot_map[i] (negative: skipped)."""
    pools = (k_codes, k_params, v_codes, v_params)
    shape = _int4_shape(k_codes)
    _slot_call("kv_write_slots_int4", slot_map, pools, (), k_new, v_new, shape,
               _int4_specs(shape, *pools[1:]), True, stream)


def kv_read_slots_fp8(slot_map, k_scale, v_scale, k_cache, v_cache, k_out, v_out, stream=None):
    """The bf16 values of the slots that slot_map names (zeros for none) of an E4M3 cache."""
    shape = _need(k_cache, torch.uint8, 4, "k_cache").shape
    _slot_call("kv_read_slots_fp8", slot_map, (k_cache, v_cache), (float(k_scale), float(v_scale)),
               k_out, v_out, shape, (("v_cache", v_cache, torch.uint8, shape),), False, stream)


def kv_read_slots_bf16(slot_map, k_cache, v_cache, k_out, v_out, stream=None):
    """The values of the slots that slot_map names (zeros for none) of a BF16 cache."""
    shape = _need(k_cache, torch.bfloat16, 4, "k_cache").shape
    _slot_call("kv_read_slots_bf16", slot_map, (k_cache, v_cache), (), k_out, v_out, shape,
               (("v_cache", v_cache, torch.bfloat16, shape),), False, stream)


def kv_read_slots_int4(slot_map, k_codes, k_params, v_codes, v_params, k_out, v_out, stream=None):
    """The bf16 values of the slots that slot_map names (zeros for none) of an INT4 cache."""
    pools = (k_codes, k_params, v_codes, v_params)
    shape = _int4_shape(k_codes)
    _slot_call("kv_read_slots_int4", slot_map, pools, (), k_out, v_out, shape,
               _int4_specs(shape, *pools[1:]), False, stream)


def kv_extend_tables(old_lens, new_lens, page_size, free_pages, num_free, page_table, slot_map,
                     cu_tokens, failed, num_free_out, num_pages, page_tags=None,
                     expected_tags=None, stream=None):
    """Grow each request from old_lens[b] to new_lens[b] tokens: take pages from the
    free stack into page_table (and their tags into expected_tags), and write the new
    tokens' slots, their packed offsets cu_tokens, the failed flags and num_free_out
    (which may be num_free)."""
    i32 = torch.int32
    B, MP = _need(page_table, i32, 2, "page_table").shape
    T = _need(slot_map, i32, 1, "slot_map").numel()
    cap = _need(free_pages, i32, 1, "free_pages").numel()
    dev, handle = _on(stream)
    _args(dev, (page_table, slot_map, free_pages), ("old_lens", old_lens, i32, (B,)),
          ("new_lens", new_lens, i32, (B,)), ("num_free", num_free, i32, (1,)),
          ("num_free_out", num_free_out, i32, (1,)), ("cu_tokens", cu_tokens, i32, (B + 1,)),
          ("failed", failed, torch.uint8, (B,)))
    if page_tags is not None or expected_tags is not None:
        if page_tags is None or expected_tags is None:
            raise ValueError("page_tags and expected_tags are given together or not at all")
        tag = _tag_dtype(page_tags, "page_tags")
        _args(dev, (), ("page_tags", page_tags, tag, (num_pages,)),
              ("expected_tags", expected_tags, tag, (B, MP)))
    _check("kv_extend_tables", _load().kv_extend_tables(
        old_lens.data_ptr(), new_lens.data_ptr(), B, _i32(page_size, "page_size"),
        free_pages.data_ptr(), cap, num_free.data_ptr(), num_free_out.data_ptr(),
        _i32(num_pages, "num_pages"), page_table.data_ptr(), MP,
        _ptr(page_tags), _ptr(expected_tags), slot_map.data_ptr(), T, cu_tokens.data_ptr(),
        failed.data_ptr(), handle))


def kv_requant_pages_fp8(src_pool, src_pages, dst_pool, dst_pages, scale, stream=None):
    """BF16 -> FP8 page handoff: page src_pages[i] -> dst_pages[i]."""
    _need(src_pool, torch.bfloat16, 4, "src_pool")
    _need(dst_pool, torch.uint8, 4, "dst_pool")
    _need(src_pages, torch.int32, 1, "src_pages")
    _need(dst_pages, torch.int32, 1, "dst_pages")
    if src_pages.shape != dst_pages.shape:
        raise ValueError("src_pages and dst_pages must have the same length")
    NPs, Hkv, P, D = src_pool.shape
    if tuple(dst_pool.shape[1:]) != (Hkv, P, D):
        raise ValueError("pools must share [Hkv][P][D]")
    _check("kv_requant_pages_fp8", _load().kv_requant_pages_fp8(
        _ptr(src_pool), NPs, _ptr(src_pages), _ptr(dst_pool), dst_pool.shape[0], _ptr(dst_pages),
        src_pages.shape[0], Hkv, P, D, float(scale), _stream(stream)))


def kv_requant_pages_int4(src_pool, src_pages, dst_codes, dst_params, dst_pages, stream=None):
    """BF16 -> INT4 page handoff: page src_pages[i] -> dst_pages[i]."""
    NPs, Hkv, P, D = _need(src_pool, torch.bfloat16, 4, "src_pool").shape
    N = _need(src_pages, torch.int32, 1, "src_pages").numel()
    NPd = _need(dst_codes, torch.uint8, 4, "dst_codes").shape[0]
    dev, handle = _on(stream)
    _args(dev, (src_pool, src_pages), ("dst_pages", dst_pages, torch.int32, (N,)),
          ("dst_codes", dst_codes, torch.uint8, (NPd, Hkv, P, D // 2)),
          ("dst_params", dst_params, torch.bfloat16, (NPd, Hkv, P, D // INT4_GROUP, 2)))
    _check("kv_requant_pages_int4", _load().kv_requant_pages_int4(
        _ptr(src_pool), NPs, _ptr(src_pages), _ptr(dst_codes), _ptr(dst_params), NPd,
        _ptr(dst_pages), N, Hkv, P, D, handle))


def paged_decode_attn_workspace_size(kv_dtype, batch, num_q_heads, num_kv_heads, head_dim,
                                     num_ctas=0) -> int:
    n = _load().paged_decode_attn_workspace_size(kv_dtype, batch, num_q_heads, num_kv_heads,
                                                 head_dim, num_ctas)
    if n == 0:
        raise PagedKVError("paged_decode_attn_workspace_size", 1,
                           _load().pkv_last_error().decode())
    return int(n)


def alloc_workspace(kv_dtype, batch, num_q_heads, num_kv_heads, head_dim, num_ctas=0,
                    device=None):
    """A uint8 CUDA tensor large enough for the attention call."""
    n = paged_decode_attn_workspace_size(kv_dtype, batch, num_q_heads, num_kv_heads, head_dim,
                                         num_ctas)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def paged_decode_attn_fp8_prefix_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                num_ctas=0):
    n = _load().paged_decode_attn_fp8_prefix_workspace_size(int(batch), int(num_q_heads),
                                                            int(num_kv_heads), int(head_dim),
                                                            int(num_ctas))
    if n == 0:
        raise PagedKVError("paged_decode_attn_fp8_prefix_workspace_size", 1,
                           _load().pkv_last_error().decode())
    return int(n)


def alloc_prefix_workspace(batch, num_q_heads, num_kv_heads, head_dim, num_ctas=0, device=None):
    """A uint8 CUDA tensor large enough for paged_decode_attn_fp8_prefix."""
    n = paged_decode_attn_fp8_prefix_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                    num_ctas)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def paged_decode_attn_plan(kv_dtype, batch, num_q_heads, num_kv_heads, head_dim, max_pages,
                           page_size, num_ctas=0):
    """The attention call's work split on the current device:
    (cluster_size, ctas, launches); cluster_size 0 means split-K + merge."""
    out = [ctypes.c_int32(0) for _ in range(3)]
    _check("paged_decode_attn_plan", _load().paged_decode_attn_plan(
        int(kv_dtype), int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim),
        int(max_pages), int(page_size), int(num_ctas), *[ctypes.byref(o) for o in out]))
    return tuple(int(o.value) for o in out)


def workspace_status(workspace) -> int:
    """The workspace status word (0 = no internal wait ever expired)."""
    return int(workspace[:4].view(torch.int32).item())


def _attn_common(q, k_cache, page_table, seq_lens, out, lse, workspace, abort):
    _need(q, torch.bfloat16, 3, "q")
    _need(page_table, torch.int32, 2, "page_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(out, torch.bfloat16, 3, "out")
    _need(lse, torch.float32, 2, "lse")
    _need(workspace, torch.uint8, 1, "workspace")
    if abort is not None:
        _need(abort, torch.uint8, 1, "abort")
    B, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    if D2 != D:
        raise ValueError("head_dim of q and cache differ")
    return B, Hq, D, NP, Hkv, P


def paged_decode_attn_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                          sm_scale, out, lse, workspace, abort=None, num_ctas=0, stream=None):
    """Decode attention over a paged E4M3 cache; writes out (bf16) and lse (fp32)."""
    _need(k_cache, torch.uint8, 4, "k_cache")
    _need(v_cache, torch.uint8, 4, "v_cache")
    B, Hq, D, NP, Hkv, P = _attn_common(q, k_cache, page_table, seq_lens, out, lse, workspace,
                                        abort)
    _check("paged_decode_attn_fp8", _load().paged_decode_attn_fp8(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale), _ptr(page_table),
        page_table.shape[1], _ptr(seq_lens), B, Hq, Hkv, D, P, NP, float(sm_scale), _ptr(abort),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), num_ctas, _stream(stream)))


def paged_decode_attn_fp8_prefix(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                 sm_scale, out, lse, workspace, abort=None, num_ctas=0,
                                 chunk_begin_out=None, stream=None):
    """paged_decode_attn_fp8 for batches whose consecutive requests share leading
    pages: the shared chunks are attended once per group.  chunk_begin_out
    (optional int32 [batch] CUDA tensor) receives, per request, the leading
    chunks attended in its tile (all of them when the tile finished it)."""
    _need(k_cache, torch.uint8, 4, "k_cache")
    _need(v_cache, torch.uint8, 4, "v_cache")
    B, Hq, D, NP, Hkv, P = _attn_common(q, k_cache, page_table, seq_lens, out, lse, workspace,
                                        abort)
    if chunk_begin_out is not None:
        _need(chunk_begin_out, torch.int32, 1, "chunk_begin_out")
        if chunk_begin_out.numel() < B:
            raise ValueError("chunk_begin_out needs batch entries")
    _check("paged_decode_attn_fp8_prefix", _load().paged_decode_attn_fp8_prefix(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale), _ptr(page_table),
        page_table.shape[1], _ptr(seq_lens), B, Hq, Hkv, D, P, NP, float(sm_scale), _ptr(abort),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), num_ctas,
        _ptr(chunk_begin_out), _stream(stream)))


def paged_decode_attn_bf16(q, k_cache, v_cache, page_table, seq_lens, sm_scale, out, lse,
                           workspace, abort=None, num_ctas=0, stream=None):
    """Decode attention over a paged BF16 cache; writes out (bf16) and lse (fp32)."""
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    B, Hq, D, NP, Hkv, P = _attn_common(q, k_cache, page_table, seq_lens, out, lse, workspace,
                                        abort)
    _check("paged_decode_attn_bf16", _load().paged_decode_attn_bf16(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1],
        _ptr(seq_lens), B, Hq, Hkv, D, P, NP, float(sm_scale), _ptr(abort), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), num_ctas, _stream(stream)))


def _attn_call(name, pools, scales, shape, specs, q, page_table, seq_lens, sm_scale, window, out,
               lse, workspace, abort, num_ctas, stream):
    """One attention call over a cache of `shape` = (NP, Hkv, P, D); pools are its
    tensors (specs: as _args takes them), scales those of FP8 pools, window the
    (window, sinks) pair or ()."""
    NP, Hkv, P, D = shape
    B, Hq, Dq = _need(q, torch.bfloat16, 3, "q").shape
    if Dq != D:
        raise ValueError("head_dim of q and cache differ")
    rows, MP = _need(page_table, torch.int32, 2, "page_table").shape
    ws = _need(workspace, torch.uint8, 1, "workspace").numel()
    dev, handle = _on(stream)
    if rows != B:
        raise ValueError(f"page_table must have a row for each of {B} requests")
    _args(dev, (q, pools[0], page_table, workspace), *specs, ("seq_lens", seq_lens, torch.int32, (B,)),
          ("out", out, torch.bfloat16, (B, Hq, D)), ("lse", lse, torch.float32, (B, Hq)))
    if abort is not None:
        _args(dev, (), ("abort", abort, torch.uint8, (B,)))
    _check(name, getattr(_load(), name)(
        q.data_ptr(), *[t.data_ptr() for t in pools], *scales, page_table.data_ptr(), MP,
        seq_lens.data_ptr(), B, Hq, Hkv, D, P, NP, float(sm_scale), *window, _ptr(abort),
        out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), ws, _i32(num_ctas, "num_ctas"), handle))


def paged_decode_attn_int4(q, k_codes, k_params, v_codes, v_params, page_table, seq_lens, sm_scale,
                           out, lse, workspace, abort=None, num_ctas=0, stream=None):
    """Decode attention over a paged INT4 cache; writes out (bf16) and lse (fp32)."""
    pools = (k_codes, k_params, v_codes, v_params)
    shape = _int4_shape(k_codes)
    _attn_call("paged_decode_attn_int4", pools, (), shape, _int4_specs(shape, *pools[1:]), q, page_table,
               seq_lens, sm_scale, (), out, lse, workspace, abort, num_ctas, stream)


def paged_decode_attn_fp8_window(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                 sm_scale, window, sinks, out, lse, workspace, abort=None,
                                 num_ctas=0, stream=None):
    """paged_decode_attn_fp8 over the last `window` and the first `sinks` tokens."""
    shape = _need(k_cache, torch.uint8, 4, "k_cache").shape
    _attn_call("paged_decode_attn_fp8_window", (k_cache, v_cache), (float(k_scale), float(v_scale)),
               shape, (("v_cache", v_cache, torch.uint8, shape),), q, page_table, seq_lens,
               sm_scale, _window(window, sinks), out, lse, workspace, abort, num_ctas, stream)


def paged_decode_attn_bf16_window(q, k_cache, v_cache, page_table, seq_lens, sm_scale, window,
                                  sinks, out, lse, workspace, abort=None, num_ctas=0, stream=None):
    """paged_decode_attn_bf16 over the last `window` and the first `sinks` tokens."""
    shape = _need(k_cache, torch.bfloat16, 4, "k_cache").shape
    _attn_call("paged_decode_attn_bf16_window", (k_cache, v_cache), (), shape,
               (("v_cache", v_cache, torch.bfloat16, shape),), q, page_table, seq_lens,
               sm_scale, _window(window, sinks), out, lse, workspace, abort, num_ctas, stream)


def paged_decode_attn_int4_window(q, k_codes, k_params, v_codes, v_params, page_table, seq_lens,
                                  sm_scale, window, sinks, out, lse, workspace, abort=None,
                                  num_ctas=0, stream=None):
    """paged_decode_attn_int4 over the last `window` and the first `sinks` tokens."""
    pools = (k_codes, k_params, v_codes, v_params)
    shape = _int4_shape(k_codes)
    _attn_call("paged_decode_attn_int4_window", pools, (), shape, _int4_specs(shape, *pools[1:]), q,
               page_table, seq_lens, sm_scale, _window(window, sinks), out, lse, workspace,
               abort, num_ctas, stream)


def paged_decode_attn_fp8_noalloc(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                  sm_scale, out, lse, abort=None, num_ctas=0, stream=None):
    """paged_decode_attn_fp8 without a workspace argument, for callers that
    cannot allocate device memory: the library uses its built-in scratch array
    (see paged_decode_attn_fp8_noalloc_scratch_bytes()).  Calls that overlap
    on the GPU share that array and must not run concurrently."""
    _need(k_cache, torch.uint8, 4, "k_cache")
    _need(v_cache, torch.uint8, 4, "v_cache")
    _need(q, torch.bfloat16, 3, "q")
    _need(page_table, torch.int32, 2, "page_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(out, torch.bfloat16, 3, "out")
    _need(lse, torch.float32, 2, "lse")
    if abort is not None:
        _need(abort, torch.uint8, 1, "abort")
    B, Hq, D = q.shape
    NP, Hkv, P, _ = k_cache.shape
    _check("paged_decode_attn_fp8_noalloc", _load().paged_decode_attn_fp8_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale), _ptr(page_table),
        page_table.shape[1], _ptr(seq_lens), B, Hq, Hkv, D, P, NP, float(sm_scale), _ptr(abort),
        _ptr(out), _ptr(lse), num_ctas, _stream(stream)))


def noalloc_scratch_bytes() -> int:
    return int(_load().paged_decode_attn_fp8_noalloc_scratch_bytes())


def noalloc_status(stream=None) -> int:
    """The built-in scratch's status word after the last no-allocation call
    on the current device (0 = no internal wait expired).  Copies 4 bytes to
    host memory on `stream` and waits for that copy."""
    import numpy as np
    word = np.zeros(1, dtype=np.uint32)
    _check("paged_decode_attn_fp8_noalloc_status", _load().paged_decode_attn_fp8_noalloc_status(
        ctypes.c_void_p(word.ctypes.data), _stream(stream)))
    (torch.cuda.current_stream() if stream is None else stream).synchronize()
    return int(word[0])


def version() -> int:
    return int(_load().pkv_version())


def int4_dequant_gemv(x, w_tiles, scales, y, group_size=128, status=None, stream=None):
    """y = x W^T with W expanded from tiled INT4 codes and per-group bf16
    scales (layouts in include/pagedkv.h; int4_tile_layout builds them)."""
    _need(x, torch.bfloat16, 2, "x")
    _need(w_tiles, torch.uint8, 4, "w_tiles")
    _need(scales, torch.bfloat16, 3, "scales")
    _need(y, torch.bfloat16, 2, "y")
    if status is not None:
        _need(status, _TAG_DTYPES, 1, "status")
    B, k = x.shape
    n = w_tiles.shape[0] * 128
    if tuple(w_tiles.shape) != (n // 128, k // 256, 128, 128) or y.shape != (B, n) or \
            k % group_size or tuple(scales.shape) != (n // 128, k // group_size, 128):
        raise ValueError("inconsistent INT4 GEMV shapes")
    _check("int4_dequant_gemv", _load().int4_dequant_gemv(
        _ptr(x), _ptr(w_tiles), _ptr(scales), B, n, k, group_size, _ptr(y), _ptr(status),
        _stream(stream)))


def int4_tile_layout(w_rowmajor, scales_rows, group_size=128):
    """Re-lay a row-major code matrix [n][k/2] (uint8, two codes per byte,
    even column in the low nibble) and row-wise scales [n][k/group_size]
    into the layouts int4_dequant_gemv reads: each 32-bit word of 8 columns
    holds the even columns in its low half-word and the odd ones in its high
    half-word, and rows are cut into 128 x 256 tiles.  Pure data movement,
    done once per weight matrix."""
    n, half = w_rowmajor.shape
    k = 2 * half
    if n % 128 or k % 256 or tuple(scales_rows.shape) != (n, k // group_size):
        raise ValueError("n must be a multiple of 128, k of 256, scales [n][k/group]")
    c = torch.stack([w_rowmajor & 0xF, w_rowmajor >> 4], dim=-1).reshape(n, k // 8, 8)
    words = torch.stack([c[..., 0] | (c[..., 2] << 4), c[..., 4] | (c[..., 6] << 4),
                         c[..., 1] | (c[..., 3] << 4), c[..., 5] | (c[..., 7] << 4)], dim=-1)
    packed = words.reshape(n, half)
    tiles = packed.reshape(n // 128, 128, k // 256, 128).permute(0, 2, 1, 3).contiguous()
    sc = scales_rows.reshape(n // 128, 128, k // group_size).permute(0, 2, 1).contiguous()
    return tiles, sc
