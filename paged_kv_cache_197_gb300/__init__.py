"""Paged KV-cache decode on GB300: Python binding of the C ABI in include/pa.h and pa_draft.h.

Every function here only marshals arguments (torch tensors -> pointers and sizes)
and calls the function of the same name in libpa.so; all of the work runs in the
library's CUDA kernels.  There is no CPU fallback: if the library is missing or
its call fails, an exception is raised.

Layouts (see include/pa.h):
  query, out        [S][Hq][D] bf16
  k_cache, v_cache  [N][Hkv][bs][D] bf16, int8, or uint8 (e4m3 codes)
  k_scale, v_scale  [N][Hkv][bs] fp32 (8-bit caches)
  block_tables      [S][M] int32, context_lens [S] int32, slot_mapping [T] int64

A step of speculative decoding over the cache (see include/pa_draft.h) is
pa_rotary_and_cache, pa_tree_attention and pa_verify_tree; rows are [T], sequence s has rows
query_start[s] .. query_start[s + 1] - 1, and parents [T] holds each row's parent in its
sequence (-1: the root).
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch

PKG = Path(__file__).resolve().parent
LIBRARY = PKG / "libpa.so"

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_OUT_OF_RANGE, PA_ERR_CUDA = range(5)
PA_KV_BF16, PA_KV_INT8, PA_KV_FP8 = 0, 1, 2
PA_FLAG_SLOT_OUT_OF_RANGE = 1
PA_FLAG_BLOCK_OUT_OF_RANGE = 2
PA_FLAG_CONTEXT_OUT_OF_RANGE = 4
PA_FLAG_PREFIX_MISMATCH = 8
PA_FLAG_QUERY_OUT_OF_RANGE = 16
PA_FLAG_TIMEOUT = 32
PA_FLAG_FP16_RANGE = 64
PA_FLAG_WORKSPACE_SHORT = 128
PA_FLAG_TREE_PARENT = 256
PA_FLAG_TOKEN_OUT_OF_RANGE = 512
PA_FLAG_PROBABILITY = 1024
PA_TREE_MAX_NODES = 256
PA_PROB_F32, PA_PROB_BF16 = 0, 1
PA_ROTARY_PLAIN, PA_ROTARY_LINEAR, PA_ROTARY_BASE, PA_ROTARY_RAMP, PA_ROTARY_WAVELENGTH = range(5)

EXPORTED = ["pa_version", "pa_status_string", "pa_last_error_string", "pa_reshape_and_cache",
            "pa_quantize_kv", "pa_quantize_kv_fp8", "pa_copy_blocks", "pa_decode_workspace_size", "pa_decode",
            "pa_decode_noalloc", "pa_decode_shared_prefix_workspace_size", "pa_decode_shared_prefix",
            "pa_multi_token_workspace_size", "pa_multi_token_workspace_size_for_tokens",
            "pa_multi_token_attention", "pa_rotary_frequencies", "pa_rotary_table", "pa_rotary_and_cache",
            "pa_tree_workspace_size", "pa_tree_attention", "pa_verify_tree"]
PA_NOALLOC_SCRATCH_BYTES = 16 << 20


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[status {status}] {message}")
        self.status = status


_LIB: ctypes.CDLL | None = None


def load_library(path: Path | str | None = None) -> ctypes.CDLL:
    """Load libpa.so (built by __graft_entry__.build()); raise if it is absent."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = Path(path) if path is not None else LIBRARY
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build the CUDA library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(str(p))
    vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float)
    lib.pa_version.restype = i32
    lib.pa_status_string.argtypes = [i32]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_last_error_string.restype = ctypes.c_char_p
    lib.pa_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_reshape_and_cache.restype = i32
    lib.pa_quantize_kv.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_quantize_kv.restype = i32
    lib.pa_quantize_kv_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_quantize_kv_fp8.restype = i32
    lib.pa_copy_blocks.argtypes = [vp, vp, vp, vp, vp, i32, i32, sz, i32, vp]
    lib.pa_copy_blocks.restype = i32
    lib.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.pa_decode_workspace_size.restype = sz
    lib.pa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                              i32, f32, i32, vp, sz, vp, vp]
    lib.pa_decode.restype = i32
    lib.pa_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32,
                                      i32, i32, f32, i32, vp, vp]
    lib.pa_decode_noalloc.restype = i32
    lib.pa_decode_shared_prefix_workspace_size.argtypes = [i32] * 9
    lib.pa_decode_shared_prefix_workspace_size.restype = sz
    lib.pa_decode_shared_prefix.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32,
                                            i32, i32, i32, f32, i32, vp, vp, i32, i32, i32, vp, sz,
                                            vp, vp]
    lib.pa_decode_shared_prefix.restype = i32
    lib.pa_multi_token_workspace_size.argtypes = [i32] * 9
    lib.pa_multi_token_workspace_size.restype = sz
    lib.pa_multi_token_workspace_size_for_tokens.argtypes = [i32] * 9 + [i64]
    lib.pa_multi_token_workspace_size_for_tokens.restype = sz
    lib.pa_multi_token_attention.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, vp, i32,
                                             i32, i32, i32, i32, i32, i32, f32, i32, i32, vp, sz,
                                             vp, vp]
    lib.pa_multi_token_attention.restype = i32
    f64 = ctypes.c_double
    lib.pa_rotary_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
    lib.pa_rotary_frequencies.restype = i32
    lib.pa_rotary_table.argtypes = [vp, i32, vp]
    lib.pa_rotary_table.restype = i32
    lib.pa_rotary_and_cache.argtypes = [vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i32, vp, vp, vp,
                                        i32, i32, f32, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_rotary_and_cache.restype = i32
    lib.pa_tree_workspace_size.argtypes = [i32] * 9
    lib.pa_tree_workspace_size.restype = sz
    lib.pa_tree_attention.argtypes = [vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, i32, vp, i32, vp, vp, vp,
                                      i32, i32, i32, i32, i32, i32, i32, f32, i32, i32, vp, sz, vp, vp]
    lib.pa_tree_attention.restype = i32
    lib.pa_verify_tree.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp, i64, i32, vp, vp, vp, vp, i32, i32, i32,
                                   i32, vp, i32, vp, i32, i32, vp, vp]
    lib.pa_verify_tree.restype = i32
    if path is None:
        _LIB = lib
    return lib


def _check(status: int) -> None:
    if status != PA_OK:
        lib = load_library()
        raise PagedAttentionError(status, lib.pa_last_error_string().decode())


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _cuda(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int | None = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got {t.dim()}")


def _stream(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _workspace(n: int, device, stream) -> torch.Tensor | None:
    """n bytes of scratch for one call on `stream`, None for none.  They are allocated on that stream:
    when the call returns they are given back, and may be used again at once by what is queued
    behind it there, but not by another stream before it has run."""
    if n == 0:
        return None
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream, device)  # (an ExternalStream of 0 would be a new stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=device)


def _flag(err_flag):
    if err_flag is not None:
        _cuda(err_flag, "err_flag", torch.int32)
    return _ptr(err_flag)


def pa_version() -> int:
    return int(load_library().pa_version())


def pa_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, err_flag=None,
                         stream=None) -> None:
    """Append the bf16 rows key/value [T][Hkv][D] into slots of a bf16 paged cache."""
    for t, n in ((key, "key"), (value, "value")):
        _cuda(t, n, torch.bfloat16, 3)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _cuda(t, n, torch.bfloat16, 4)
    _cuda(slot_mapping, "slot_mapping", torch.int64, 1)
    T, Hkv, D = key.shape
    N, Hkv2, bs, D2 = k_cache.shape
    if value.shape != key.shape or v_cache.shape != k_cache.shape or (Hkv2, D2) != (Hkv, D) \
            or slot_mapping.shape[0] != T:
        raise ValueError("pa_reshape_and_cache: shape mismatch")
    lib = load_library()
    _check(lib.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(slot_mapping), T, Hkv, D, bs, N, _flag(err_flag),
                                    _stream(stream, key.device)))


def pa_quantize_kv(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, err_flag=None,
                   stream=None) -> None:
    """Quantise bf16 rows [T][Hkv][D] to int8 with a per-(token, kv head) scale and append."""
    for t, n in ((key, "key"), (value, "value")):
        _cuda(t, n, torch.bfloat16, 3)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _cuda(t, n, torch.int8, 4)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _cuda(t, n, torch.float32, 3)
    _cuda(slot_mapping, "slot_mapping", torch.int64, 1)
    T, Hkv, D = key.shape
    N, Hkv2, bs, D2 = k_cache.shape
    if value.shape != key.shape or v_cache.shape != k_cache.shape or (Hkv2, D2) != (Hkv, D) \
            or tuple(k_scale.shape) != (N, Hkv, bs) or v_scale.shape != k_scale.shape \
            or slot_mapping.shape[0] != T:
        raise ValueError("pa_quantize_kv: shape mismatch")
    lib = load_library()
    _check(lib.pa_quantize_kv(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                              _ptr(v_scale), _ptr(slot_mapping), T, Hkv, D, bs, N, _flag(err_flag),
                              _stream(stream, key.device)))


FP8_DTYPES = (torch.uint8,) + ((torch.float8_e4m3fn,) if hasattr(torch, "float8_e4m3fn") else ())


def kv_dtype_of(cache: torch.Tensor) -> int:
    """PA_KV_* code of a cache tensor: bf16, int8, or fp8 e4m3 bytes (uint8 or float8_e4m3fn)."""
    if cache.dtype == torch.bfloat16:
        return PA_KV_BF16
    if cache.dtype == torch.int8:
        return PA_KV_INT8
    if cache.dtype in FP8_DTYPES:
        return PA_KV_FP8
    raise TypeError(f"unsupported cache dtype {cache.dtype}")


def pa_quantize_kv_fp8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, err_flag=None,
                       stream=None) -> None:
    """Quantise bf16 rows [T][Hkv][D] to fp8 e4m3 with a per-(token, kv head) scale and append."""
    for t, n in ((key, "key"), (value, "value")):
        _cuda(t, n, torch.bfloat16, 3)
    if k_cache.dtype not in FP8_DTYPES:
        raise TypeError("fp8 caches are uint8 or float8_e4m3fn tensors")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _cuda(t, n, k_cache.dtype, 4)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _cuda(t, n, torch.float32, 3)
    _cuda(slot_mapping, "slot_mapping", torch.int64, 1)
    T, Hkv, D = key.shape
    N, Hkv2, bs, D2 = k_cache.shape
    if value.shape != key.shape or v_cache.shape != k_cache.shape or (Hkv2, D2) != (Hkv, D) \
            or tuple(k_scale.shape) != (N, Hkv, bs) or v_scale.shape != k_scale.shape \
            or slot_mapping.shape[0] != T:
        raise ValueError("pa_quantize_kv_fp8: shape mismatch")
    lib = load_library()
    _check(lib.pa_quantize_kv_fp8(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                  _ptr(v_scale), _ptr(slot_mapping), T, Hkv, D, bs, N, _flag(err_flag),
                                  _stream(stream, key.device)))


def pa_copy_blocks(k_cache, v_cache, block_mapping, k_scale=None, v_scale=None,
                   stream=None) -> None:
    """Copy whole physical blocks (src, dst) of both caches (and scales, if given).

    block_mapping is a HOST sequence of (src, dst) pairs (tensor, ndarray or list)."""
    kv_dtype_of(k_cache)
    _cuda(k_cache, "k_cache", k_cache.dtype)
    _cuda(v_cache, "v_cache", k_cache.dtype)
    if v_cache.shape != k_cache.shape:
        raise ValueError("pa_copy_blocks: cache shapes differ")
    pairs = torch.as_tensor(block_mapping, dtype=torch.int64, device="cpu").reshape(-1, 2).contiguous()
    N = k_cache.shape[0]
    block_bytes = k_cache.numel() * k_cache.element_size() // N
    scale_elems = 0
    if k_scale is not None or v_scale is not None:
        if k_scale is None or v_scale is None:
            raise ValueError("give both scale arrays or neither")
        _cuda(k_scale, "k_scale", torch.float32)
        _cuda(v_scale, "v_scale", torch.float32)
        if k_scale.shape[0] != N or v_scale.shape != k_scale.shape:
            raise ValueError("pa_copy_blocks: scale shapes")
        scale_elems = k_scale.numel() // N
    lib = load_library()
    _check(lib.pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                              pairs.data_ptr(), pairs.shape[0], N, block_bytes, scale_elems,
                              _stream(stream, k_cache.device)))


def pa_decode_workspace_size(S: int, Hq: int, Hkv: int, D: int, bs: int, kv_dtype: int,
                             max_context_len: int) -> int:
    return int(load_library().pa_decode_workspace_size(S, Hq, Hkv, D, bs, kv_dtype,
                                                       max_context_len))


def pa_decode(out, query, k_cache, v_cache, block_tables, context_lens, scale: float,
              max_context_len: int, workspace=None, k_scale=None, v_scale=None, err_flag=None,
              stream=None) -> None:
    """Paged decode attention; writes out [S][Hq][D] bf16."""
    _cuda(out, "out", torch.bfloat16, 3)
    _cuda(query, "query", torch.bfloat16, 3)
    kv_dtype = kv_dtype_of(k_cache)
    _cuda(k_cache, "k_cache", k_cache.dtype, 4)
    _cuda(v_cache, "v_cache", k_cache.dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    if kv_dtype != PA_KV_BF16:
        if k_scale is None or v_scale is None:
            raise ValueError("an int8 or fp8 cache needs k_scale and v_scale")
        _cuda(k_scale, "k_scale", torch.float32, 3)
        _cuda(v_scale, "v_scale", torch.float32, 3)
    S, Hq, D = query.shape
    N, Hkv, bs, D2 = k_cache.shape
    M = block_tables.shape[1]
    if out.shape != query.shape or v_cache.shape != k_cache.shape or D2 != D \
            or block_tables.shape[0] != S or context_lens.shape[0] != S:
        raise ValueError("pa_decode: shape mismatch")
    ws_bytes = 0
    if workspace is not None:
        _cuda(workspace, "workspace", workspace.dtype)
        ws_bytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    _check(lib.pa_decode(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                         _ptr(v_scale), kv_dtype, _ptr(block_tables), M, _ptr(context_lens), S, Hq,
                         Hkv, D, bs, N, float(scale), int(max_context_len), _ptr(workspace),
                         ws_bytes, _flag(err_flag), _stream(stream, query.device)))


def pa_decode_noalloc(out, query, k_cache, v_cache, block_tables, context_lens, scale: float,
                      max_context_len: int, k_scale=None, v_scale=None, err_flag=None,
                      stream=None) -> None:
    """pa_decode for callers that cannot allocate: the library's own fixed scratch array
    (PA_NOALLOC_SCRATCH_BYTES per GPU) replaces the workspace.  Calls sharing a device
    must not overlap on the GPU."""
    _cuda(out, "out", torch.bfloat16, 3)
    _cuda(query, "query", torch.bfloat16, 3)
    kv_dtype = kv_dtype_of(k_cache)
    _cuda(k_cache, "k_cache", k_cache.dtype, 4)
    _cuda(v_cache, "v_cache", k_cache.dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    if kv_dtype != PA_KV_BF16:
        if k_scale is None or v_scale is None:
            raise ValueError("an int8 or fp8 cache needs k_scale and v_scale")
        _cuda(k_scale, "k_scale", torch.float32, 3)
        _cuda(v_scale, "v_scale", torch.float32, 3)
    S, Hq, D = query.shape
    N, Hkv, bs, D2 = k_cache.shape
    if out.shape != query.shape or v_cache.shape != k_cache.shape or D2 != D \
            or block_tables.shape[0] != S or context_lens.shape[0] != S:
        raise ValueError("pa_decode_noalloc: shape mismatch")
    lib = load_library()
    _check(lib.pa_decode_noalloc(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(k_scale), _ptr(v_scale), kv_dtype, _ptr(block_tables),
                                 block_tables.shape[1], _ptr(context_lens), S, Hq, Hkv, D, bs, N,
                                 float(scale), int(max_context_len), _flag(err_flag),
                                 _stream(stream, query.device)))


def pa_decode_shared_prefix_workspace_size(S: int, Hq: int, Hkv: int, D: int, bs: int,
                                           kv_dtype: int, max_context_len: int,
                                           max_group_size: int, max_prefix_len: int) -> int:
    return int(load_library().pa_decode_shared_prefix_workspace_size(
        S, Hq, Hkv, D, bs, kv_dtype, max_context_len, max_group_size, max_prefix_len))


def pa_decode_shared_prefix(out, query, k_cache, v_cache, block_tables, context_lens,
                            scale: float, max_context_len: int, group_start, group_prefix_len,
                            max_group_size: int, max_prefix_len: int, workspace=None,
                            k_scale=None, v_scale=None, err_flag=None, stream=None) -> None:
    """Paged decode of a batch whose groups of consecutive sequences share prefix blocks;
    the same result as pa_decode.  group_start [n_groups + 1] and group_prefix_len
    [n_groups] are int32 device tensors; workspace defaults to a fresh allocation."""
    _cuda(out, "out", torch.bfloat16, 3)
    _cuda(query, "query", torch.bfloat16, 3)
    kv_dtype = kv_dtype_of(k_cache)
    _cuda(k_cache, "k_cache", k_cache.dtype, 4)
    _cuda(v_cache, "v_cache", k_cache.dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    _cuda(group_start, "group_start", torch.int32, 1)
    _cuda(group_prefix_len, "group_prefix_len", torch.int32, 1)
    if kv_dtype != PA_KV_BF16:
        if k_scale is None or v_scale is None:
            raise ValueError("an int8 or fp8 cache needs k_scale and v_scale")
        _cuda(k_scale, "k_scale", torch.float32, 3)
        _cuda(v_scale, "v_scale", torch.float32, 3)
    S, Hq, D = query.shape
    N, Hkv, bs, D2 = k_cache.shape
    M = block_tables.shape[1]
    n_groups = group_prefix_len.shape[0]
    if out.shape != query.shape or v_cache.shape != k_cache.shape or D2 != D \
            or block_tables.shape[0] != S or context_lens.shape[0] != S \
            or group_start.shape[0] != n_groups + 1:
        raise ValueError("pa_decode_shared_prefix: shape mismatch")
    if workspace is None:
        n = pa_decode_shared_prefix_workspace_size(S, Hq, Hkv, D, bs, kv_dtype, max_context_len,
                                                   max_group_size, max_prefix_len)
        workspace = _workspace(max(n, 1), query.device, stream)
    _cuda(workspace, "workspace", workspace.dtype)
    ws_bytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    _check(lib.pa_decode_shared_prefix(
        _ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
        kv_dtype, _ptr(block_tables), M, _ptr(context_lens), S, Hq, Hkv, D, bs, N, float(scale),
        int(max_context_len), _ptr(group_start), _ptr(group_prefix_len), n_groups,
        int(max_group_size), int(max_prefix_len), _ptr(workspace), ws_bytes, _flag(err_flag),
        _stream(stream, query.device)))


def pa_multi_token_workspace_size(S: int, T: int, Hq: int, Hkv: int, D: int, bs: int,
                                  kv_dtype: int, max_context_len: int, max_query_len: int) -> int:
    return int(load_library().pa_multi_token_workspace_size(
        S, T, Hq, Hkv, D, bs, kv_dtype, max_context_len, max_query_len))


def pa_multi_token_workspace_size_for_tokens(S: int, T: int, Hq: int, Hkv: int, D: int, bs: int,
                                             kv_dtype: int, max_context_len: int, max_query_len: int,
                                             total_context_tokens: int) -> int:
    return int(load_library().pa_multi_token_workspace_size_for_tokens(
        S, T, Hq, Hkv, D, bs, kv_dtype, max_context_len, max_query_len, int(total_context_tokens)))


def pa_multi_token_attention(out, query, k_cache, v_cache, block_tables, context_lens,
                             query_start, scale: float, max_context_len: int,
                             max_query_len: int, workspace=None, k_scale=None, v_scale=None,
                             err_flag=None, stream=None, total_context_tokens=None) -> None:
    """Several new tokens per sequence attend the paged cache, each up to its own
    position: query/out [T][Hq][D] bf16, sequence s owning rows
    query_start[s] .. query_start[s+1]-1.  workspace defaults to a fresh allocation."""
    _cuda(out, "out", torch.bfloat16, 3)
    _cuda(query, "query", torch.bfloat16, 3)
    kv_dtype = kv_dtype_of(k_cache)
    _cuda(k_cache, "k_cache", k_cache.dtype, 4)
    _cuda(v_cache, "v_cache", k_cache.dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    _cuda(query_start, "query_start", torch.int32, 1)
    if kv_dtype != PA_KV_BF16:
        if k_scale is None or v_scale is None:
            raise ValueError("an int8 or fp8 cache needs k_scale and v_scale")
        _cuda(k_scale, "k_scale", torch.float32, 3)
        _cuda(v_scale, "v_scale", torch.float32, 3)
    T, Hq, D = query.shape
    N, Hkv, bs, D2 = k_cache.shape
    S = context_lens.shape[0]
    M = block_tables.shape[1]
    if out.shape != query.shape or v_cache.shape != k_cache.shape or D2 != D \
            or block_tables.shape[0] != S or query_start.shape[0] != S + 1:
        raise ValueError("pa_multi_token_attention: shape mismatch")
    if workspace is None:
        if total_context_tokens is None:
            n = pa_multi_token_workspace_size(S, T, Hq, Hkv, D, bs, kv_dtype, max_context_len,
                                              max_query_len)
        else:
            n = pa_multi_token_workspace_size_for_tokens(S, T, Hq, Hkv, D, bs, kv_dtype,
                                                         max_context_len, max_query_len,
                                                         total_context_tokens)
        workspace = _workspace(n, query.device, stream)
    ws_bytes = 0
    if workspace is not None:
        _cuda(workspace, "workspace", workspace.dtype)
        ws_bytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    _check(lib.pa_multi_token_attention(
        _ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
        kv_dtype, _ptr(block_tables), M, _ptr(context_lens), _ptr(query_start), S, T, Hq, Hkv, D, bs, N,
        float(scale), int(max_context_len), int(max_query_len), _ptr(workspace), ws_bytes,
        _flag(err_flag), _stream(stream, query.device)))


def decode_workspace(query, k_cache, max_context_len: int) -> torch.Tensor | None:
    """Allocate (with torch) the scratch pa_decode needs for these shapes, or None."""
    S, Hq, D = query.shape
    N, Hkv, bs, _ = k_cache.shape
    kv_dtype = kv_dtype_of(k_cache)
    n = pa_decode_workspace_size(S, Hq, Hkv, D, bs, kv_dtype, max_context_len)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=query.device)


# ------------------------------------------------- speculative decoding (include/pa_draft.h)
# These calls are short, so their checks are kept short as well: one pass over a tensor's
# properties that gives its address, and the named error only where something is wrong.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _need(t, name: str, dtype: torch.dtype, ndim: int, index: int) -> int:
    """Address of a contiguous tensor of this type on device `index`."""
    if t.dtype is dtype and t.get_device() == index and t.dim() == ndim and t.is_contiguous():
        return t.data_ptr()
    _cuda(t, name, dtype, ndim)
    raise ValueError(f"{name}: all tensors must live on one CUDA device")


def _heads(t, name: str, index: int) -> int:
    """Token stride, in elements, of a [T][heads][D] bf16 tensor with dense heads on device `index`."""
    if t.dtype is torch.bfloat16 and t.get_device() == index and t.dim() == 3:
        _, heads, D = t.shape
        by_token, by_head, by_element = t.stride()
        if (by_element == 1 or D <= 1) and (by_head == D or heads <= 1):
            return by_token if t.shape[0] > 1 else heads * D
        raise ValueError(f"{name}: the heads of a token must be dense")
    if t.is_contiguous():
        _cuda(t, name, torch.bfloat16, 3)
    elif t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    elif t.dim() != 3:
        raise ValueError(f"{name}: expected 3 dimensions, got {t.dim()}")
    raise ValueError(f"{name}: all tensors must live on one CUDA device")


def _first_device(t, name: str) -> int:
    """Index of the CUDA device a call runs on: that of its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    return t.get_device()


def _scales(k_scale, v_scale, N: int, Hkv: int, bs: int, kv_dtype: int, index: int, fn: str):
    """Addresses of an 8-bit cache's scales; (None, None) for a bf16 cache."""
    if kv_dtype == PA_KV_BF16:
        return None, None
    if k_scale is None or v_scale is None:
        raise ValueError("an int8 or fp8 cache needs k_scale and v_scale")
    ks, vs = _need(k_scale, "k_scale", torch.float32, 3, index), _need(v_scale, "v_scale", torch.float32, 3, index)
    if tuple(k_scale.shape) != (N, Hkv, bs) or v_scale.shape != k_scale.shape:
        raise ValueError(f"{fn}: scale shapes")
    return ks, vs


def _call(function, index: int, stream, *args) -> None:
    """Call a library function with device `index` current and the stream as its last argument."""
    if stream is None and _raw_stream is not None:
        raw = _raw_stream(index)
    else:
        raw = _stream(stream, index)
    if torch.cuda.current_device() == index:
        status = function(*args, raw)
    else:
        with torch.cuda.device(index):
            status = function(*args, raw)
    if status != PA_OK:
        _check(status)


def pa_rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = PA_ROTARY_PLAIN, factor: float = 1.0,
                          original_context: float = 0.0, p0: float = 0.0, p1: float = 0.0):
    """(inv_freq [rot_dim / 2] float64 on the host, attention_factor) of a scaling rule."""
    inv = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.float64)
    attention = ctypes.c_double(1.0)
    _check(load_library().pa_rotary_frequencies(int(rot_dim), float(base), int(scaling), float(factor),
                                                float(original_context), float(p0), float(p1), inv.data_ptr(),
                                                ctypes.byref(attention)))
    return inv, attention.value


def pa_rotary_table(inv_freq, device=None) -> torch.Tensor:
    """The 64-bit table of host frequencies (radians per position), as int64 bit patterns on
    `device`."""
    inv = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").contiguous()
    if inv.dim() != 1:
        raise ValueError("inv_freq: expected 1 dimension")
    table = torch.empty(inv.shape[0], dtype=torch.int64)
    _check(load_library().pa_rotary_table(inv.data_ptr(), inv.shape[0], table.data_ptr()))
    return table if device is None else table.to(device)


def pa_rotary_and_cache(query_out, query, key, positions, table, interleaved: bool = False,
                        attention_factor: float = 1.0, key_out=None, value=None, k_cache=None, v_cache=None,
                        slot_mapping=None, k_scale=None, v_scale=None, err_flag=None, stream=None) -> None:
    """Rotate query [T][Hq][D] and key [T][Hkv][D] to positions [T] (int64), the first
    2 * len(table) elements of each head; write query_out, key_out if given, and append the
    rotated keys and the values if a cache is given.  query, key and value may be slices of
    one tensor (dense heads, any token stride that is a multiple of 8)."""
    dev = _first_device(query, "query")
    q_stride, k_stride = _heads(query, "query", dev), _heads(key, "key", dev)
    T, Hq, D = query.shape
    T2, Hkv, D2 = key.shape
    qo = _need(query_out, "query_out", torch.bfloat16, 3, dev)
    pos = _need(positions, "positions", torch.int64, 1, dev)
    tab = _need(table, "table", torch.int64, 1, dev)
    if query_out.shape != query.shape or T2 != T or D2 != D or positions.shape[0] != T:
        raise ValueError("pa_rotary_and_cache: shape mismatch")
    ko = None
    if key_out is not None:
        ko = _need(key_out, "key_out", torch.bfloat16, 3, dev)
        if key_out.shape != key.shape:
            raise ValueError("pa_rotary_and_cache: shape mismatch")
    v_stride, kv_dtype, bs, N = 0, PA_KV_BF16, 16, 1
    vp = kc = vc = ks = vs = slots = None
    if k_cache is not None or v_cache is not None:
        if k_cache is None or v_cache is None or value is None or slot_mapping is None:
            raise ValueError("appending needs k_cache, v_cache, value and slot_mapping")
        v_stride, vp, kv_dtype = _heads(value, "value", dev), value.data_ptr(), kv_dtype_of(k_cache)
        kc = _need(k_cache, "k_cache", k_cache.dtype, 4, dev)
        vc = _need(v_cache, "v_cache", k_cache.dtype, 4, dev)
        slots = _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
        shape = k_cache.shape
        N, heads, bs, D2 = shape
        if value.shape != key.shape or v_cache.shape != shape or heads != Hkv or D2 != D or slot_mapping.shape[0] != T:
            raise ValueError("pa_rotary_and_cache: shape mismatch")
        ks, vs = _scales(k_scale, v_scale, N, Hkv, bs, kv_dtype, dev, "pa_rotary_and_cache")
    flag = None if err_flag is None else _need(err_flag, "err_flag", torch.int32, err_flag.dim(), dev)
    _call(load_library().pa_rotary_and_cache, dev, stream, qo, ko, query.data_ptr(), q_stride, key.data_ptr(), k_stride,
          vp, v_stride, kc, vc, ks, vs, kv_dtype, slots, pos, tab, 2 * table.shape[0], 1 if interleaved else 0,
          attention_factor, T, Hq, Hkv, D, bs, N, flag)


def pa_tree_workspace_size(S: int, T: int, Hq: int, Hkv: int, D: int, bs: int, kv_dtype: int,
                           max_context_len: int, max_query_len: int) -> int:
    return int(load_library().pa_tree_workspace_size(S, T, Hq, Hkv, D, bs, kv_dtype, max_context_len,
                                                     max_query_len))


def pa_tree_attention(out, query, key, value, k_cache, v_cache, block_tables, context_lens, query_start, parents,
                      scale: float, max_context_len: int, max_query_len: int, workspace=None, k_scale=None,
                      v_scale=None, err_flag=None, stream=None) -> None:
    """Rows of drafted tokens attend their sequence's cached context and, among the rows
    (key/value [T][Hkv][D] beside the cache), themselves and their ancestors.  workspace
    defaults to a fresh allocation."""
    dev = _first_device(query, "query")
    qp = _need(query, "query", torch.bfloat16, 3, dev)
    op = _need(out, "out", torch.bfloat16, 3, dev)
    k_stride, v_stride, kv_dtype = _heads(key, "key", dev), _heads(value, "value", dev), kv_dtype_of(k_cache)
    kc = _need(k_cache, "k_cache", k_cache.dtype, 4, dev)
    vc = _need(v_cache, "v_cache", k_cache.dtype, 4, dev)
    tables = _need(block_tables, "block_tables", torch.int32, 2, dev)
    lens = _need(context_lens, "context_lens", torch.int32, 1, dev)
    starts = _need(query_start, "query_start", torch.int32, 1, dev)
    up = _need(parents, "parents", torch.int32, 1, dev)
    shape, cache_shape = query.shape, k_cache.shape
    T, Hq, D = shape
    N, Hkv, bs, D2 = cache_shape
    S, M = block_tables.shape
    ks, vs = _scales(k_scale, v_scale, N, Hkv, bs, kv_dtype, dev, "pa_tree_attention")
    if out.shape != shape or key.shape != (T, Hkv, D) or value.shape != key.shape or v_cache.shape != cache_shape \
            or D2 != D or context_lens.shape[0] != S or query_start.shape[0] != S + 1 or parents.shape[0] != T:
        raise ValueError("pa_tree_attention: shape mismatch")
    if workspace is None:
        n = pa_tree_workspace_size(S, T, Hq, Hkv, D, bs, kv_dtype, max_context_len, max_query_len)
        workspace = _workspace(n, query.device, stream)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws = _need(workspace, "workspace", workspace.dtype, workspace.dim(), dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    flag = None if err_flag is None else _need(err_flag, "err_flag", torch.int32, err_flag.dim(), dev)
    _call(load_library().pa_tree_attention, dev, stream, op, qp, key.data_ptr(), k_stride, value.data_ptr(), v_stride, kc,
          vc, ks, vs, kv_dtype, tables, M, lens, starts, up, S, T, Hq, Hkv, D, bs, N, scale, max_context_len,
          max_query_len, ws, ws_bytes, flag)


def _probabilities(t, name: str, T: int, V: int, dtype: torch.dtype, index: int) -> int:
    """Row stride, in elements, of [T][V] probabilities with dense rows on device `index`."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must live on the CUDA device of the other tensors")
    if t.shape != (T, V):
        raise ValueError(f"{name}: expected shape {(T, V)}, got {tuple(t.shape)}")
    by_row, by_entry = t.stride()
    if V > 1 and by_entry != 1:
        raise ValueError(f"{name}: the probabilities of a row must be dense")
    return by_row if T > 1 else V


def pa_verify_tree(tokens_out, path, n_out, draft_tokens, target_probs, query_start, parents, uniforms,
                   final_uniforms, draft_probs=None, slot_mapping=None, block_tables=None, context_lens=None,
                   block_size: int = 16, num_blocks: int = 0, err_flag=None, stream=None) -> None:
    """Accept or reject drafted tokens against target_probs [T][V] (fp32 or bf16) with given
    uniform numbers, draw each sequence's next token, and write the accepted branch: tokens_out
    and path [S][max_query_len], n_out [S], and (with block_tables, context_lens, block_size
    and num_blocks) slot_mapping [T]."""
    dev = _first_device(target_probs, "target_probs")
    said = _need(tokens_out, "tokens_out", torch.int32, 2, dev)
    way = _need(path, "path", torch.int32, 2, dev)
    count = _need(n_out, "n_out", torch.int32, 1, dev)
    tokens = _need(draft_tokens, "draft_tokens", torch.int32, 1, dev)
    starts = _need(query_start, "query_start", torch.int32, 1, dev)
    up = _need(parents, "parents", torch.int32, 1, dev)
    u = _need(uniforms, "uniforms", torch.float32, 1, dev)
    u_final = _need(final_uniforms, "final_uniforms", torch.float32, 1, dev)
    T, S = draft_tokens.shape[0], n_out.shape[0]
    dtype = target_probs.dtype
    if target_probs.dim() != 2:
        raise ValueError("target_probs: expected 2 dimensions")
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError("target_probs: expected float32 or bfloat16")
    V = target_probs.shape[1]
    p_stride = _probabilities(target_probs, "target_probs", T, V, dtype, dev)
    qp, q_stride = None, 0
    if draft_probs is not None:
        if draft_probs.dim() != 2:
            raise ValueError("draft_probs: expected 2 dimensions")
        qp, q_stride = draft_probs.data_ptr(), _probabilities(draft_probs, "draft_probs", T, V, dtype, dev)
    shape = tokens_out.shape
    W = shape[1]
    if shape[0] != S or path.shape != shape or query_start.shape[0] != S + 1 or parents.shape[0] != T \
            or uniforms.shape[0] != T or final_uniforms.shape[0] != S:
        raise ValueError("pa_verify_tree: shape mismatch")
    M, slots, tables, lens = 0, None, None, None
    if slot_mapping is not None:
        if block_tables is None or context_lens is None:
            raise ValueError("slot_mapping needs block_tables and context_lens")
        slots = _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
        tables = _need(block_tables, "block_tables", torch.int32, 2, dev)
        lens = _need(context_lens, "context_lens", torch.int32, 1, dev)
        if slot_mapping.shape[0] != T or block_tables.shape[0] != S or context_lens.shape[0] != S:
            raise ValueError("pa_verify_tree: shape mismatch")
        M = block_tables.shape[1]
    flag = None if err_flag is None else _need(err_flag, "err_flag", torch.int32, err_flag.dim(), dev)
    _call(load_library().pa_verify_tree, dev, stream, said, way, count, slots, tokens, target_probs.data_ptr(), p_stride,
          qp, q_stride, PA_PROB_F32 if dtype is torch.float32 else PA_PROB_BF16, starts, up, u, u_final, S, T, V, W,
          tables, M, lens, block_size, num_blocks, flag)


# ------------------------------------------------------------------ block manager
PA_ERR_NO_SPACE = 5
BLOCK_MANAGER_EXPORTED = ["pa_bm_create", "pa_bm_destroy", "pa_bm_add_sequence", "pa_bm_append",
                          "pa_bm_fork", "pa_bm_free", "pa_bm_block_table", "pa_bm_get_stats"]


class BlockManagerStats(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int64) for name in (
        "num_blocks", "free_blocks", "cached_blocks", "used_blocks", "used_slots", "cow_copies",
        "prefix_lookup_blocks", "prefix_hit_blocks", "evictions")]

    def as_dict(self) -> dict:
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


def _bm_lib() -> ctypes.CDLL:
    lib = load_library()
    if not getattr(lib, "_bm_ready", False):
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        lib.pa_bm_create.argtypes = [i32, i32, ctypes.POINTER(vp)]
        lib.pa_bm_create.restype = i32
        lib.pa_bm_destroy.argtypes = [vp]
        lib.pa_bm_destroy.restype = None
        lib.pa_bm_add_sequence.argtypes = [vp, i64, vp, i32, ctypes.POINTER(i32)]
        lib.pa_bm_add_sequence.restype = i32
        lib.pa_bm_append.argtypes = [vp, i64, vp, i32, vp, vp, i32, ctypes.POINTER(i32)]
        lib.pa_bm_append.restype = i32
        lib.pa_bm_fork.argtypes = [vp, i64, i64]
        lib.pa_bm_fork.restype = i32
        lib.pa_bm_free.argtypes = [vp, i64]
        lib.pa_bm_free.restype = i32
        lib.pa_bm_block_table.argtypes = [vp, i64, vp, i32, ctypes.POINTER(i32), ctypes.POINTER(i64)]
        lib.pa_bm_block_table.restype = i32
        lib.pa_bm_get_stats.argtypes = [vp, ctypes.POINTER(BlockManagerStats)]
        lib.pa_bm_get_stats.restype = i32
        lib._bm_ready = True
    return lib


class BlockManager:
    """Host block manager of include/pa_blocks.h (pool, tables, copy-on-write, prefix
    cache, LRU eviction).  Token ids and slots are plain Python ints / lists."""

    def __init__(self, num_blocks: int, block_size: int):
        self._lib = _bm_lib()
        self._h = ctypes.c_void_p()
        _check(self._lib.pa_bm_create(num_blocks, block_size, ctypes.byref(self._h)))
        self.num_blocks, self.block_size = num_blocks, block_size

    def close(self):
        if self._h:
            self._lib.pa_bm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    @staticmethod
    def _ids(tokens):
        if tokens is None:
            return None, 0
        arr = (ctypes.c_int32 * len(tokens))(*tokens)
        return arr, len(tokens)

    def add_sequence(self, seq_id: int, prompt=None) -> int:
        """Register a sequence; returns the number of prompt tokens found cached."""
        arr, n = self._ids(prompt)
        cached = ctypes.c_int(0)
        _check(self._lib.pa_bm_add_sequence(self._h, seq_id, arr, n, ctypes.byref(cached)))
        return cached.value

    def append(self, seq_id: int, n: int | None = None, tokens=None):
        """Append tokens (ids optional); returns (slots, cow_pairs)."""
        if tokens is not None:
            n = len(tokens)
        arr, _ = self._ids(tokens)
        slots = (ctypes.c_int64 * max(n, 1))()
        cow = (ctypes.c_int64 * 2)()
        n_cow = ctypes.c_int(0)
        _check(self._lib.pa_bm_append(self._h, seq_id, arr, n, slots, cow, 1, ctypes.byref(n_cow)))
        pairs = [(cow[0], cow[1])] if n_cow.value else []
        return list(slots)[:n], pairs

    def fork(self, parent: int, child: int) -> None:
        _check(self._lib.pa_bm_fork(self._h, parent, child))

    def free(self, seq_id: int) -> None:
        _check(self._lib.pa_bm_free(self._h, seq_id))

    def block_table(self, seq_id: int):
        n = ctypes.c_int(0)
        length = ctypes.c_int64(0)
        _check(self._lib.pa_bm_block_table(self._h, seq_id, None, 0, ctypes.byref(n), ctypes.byref(length)))
        table = (ctypes.c_int32 * max(n.value, 1))()
        _check(self._lib.pa_bm_block_table(self._h, seq_id, table, n.value, ctypes.byref(n),
                                           ctypes.byref(length)))
        return list(table)[: n.value], length.value

    def stats(self) -> dict:
        out = BlockManagerStats()
        _check(self._lib.pa_bm_get_stats(self._h, ctypes.byref(out)))
        return out.as_dict()
