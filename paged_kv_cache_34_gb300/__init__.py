"""Attention over a paged KV cache on NVIDIA GB300 (sm_103a).

Python binding of ``libpa.so``, the C-ABI CUDA library declared in
``include/pa.h``.  Each function here only marshals torch tensors into the
C call (device pointers, sizes, strides, the current CUDA stream) and turns a
non-OK status into an exception; every step of the computation runs in the
library's kernels.  There is no CPU fallback: without the built library the
first call raises.

    pa_reshape_and_cache  new K/V rows -> pool rows given by slot_mapping
    pa_rope_and_cache     norm and rotation of query and key heads, and the cache write
    pa_qk_norm_rope       the same without a cache
    pa_decode             one query per sequence, split-KV + LSE combine
    pa_prefill_varlen     causal attention for cu_seqlens-packed queries
    pa_reshape_and_cache_int8, pa_decode_int8, pa_decode_write_int8 (and _fp8)
                          the write, decode and step over INT8 (FP8 E4M3) pools
    pa_reshape_and_cache_fp4, pa_decode_fp4, pa_decode_write_fp4
                          the same over 4-bit pools (E2M1 codes, E4M3 group scales)
    pa_gather_cache_fp4   4-bit pools read back as 16-bit rows
    pa_copy_blocks        copy whole blocks of both pools (copy-on-write)
    pa_build_tables       a step's block tables, slots, positions and cumulative
                          lengths from request lengths
    pa_attention_varlen   causal attention of packed prompts from their K/V rows
    pa_decode_shared      decode of a batch whose groups share a prefix

Build the library with ``python -m paged_kv_cache_34_gb300.build``.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = ["pa_reshape_and_cache", "pa_rope_and_cache", "pa_qk_norm_rope", "pa_decode", "pa_decode_plan", "pa_decode_write",
           "pa_prefill_varlen", "pa_reshape_and_cache_int8", "pa_decode_int8",
           "pa_decode_write_int8", "pa_reshape_and_cache_fp8", "pa_decode_fp8",
           "pa_decode_write_fp8", "pa_reshape_and_cache_fp4", "pa_gather_cache_fp4",
           "pa_decode_fp4", "pa_decode_fp4_plan", "pa_decode_write_fp4", "pa_copy_blocks", "pa_build_tables",
           "pa_attention_varlen", "pa_decode_shared", "pa_decode_shared_plan", "PaError",
           "library", "DEVERR_SLOT", "DEVERR_BLOCK_ID", "DEVERR_CU_SEQLENS",
           "DEVERR_CONTEXT", "DEVERR_TIMEOUT", "DEVERR_SCALE", "DEVERR_NO_BLOCKS",
           "DEVERR_POSITION", "LIB_PATH"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpa.so")

# Device error bits (include/pa.h PA_DEVERR_*).
DEVERR_SLOT, DEVERR_BLOCK_ID, DEVERR_CU_SEQLENS, DEVERR_CONTEXT, DEVERR_TIMEOUT = 1, 2, 4, 8, 16
DEVERR_SCALE = 32
DEVERR_NO_BLOCKS = 64
DEVERR_POSITION = 128

_STATUS = {0: "PA_OK", 1: "PA_ERR_NULL", 2: "PA_ERR_SHAPE", 3: "PA_ERR_UNSUPPORTED",
           4: "PA_ERR_ALIGN", 5: "PA_ERR_WORKSPACE", 6: "PA_ERR_CUDA"}
_DTYPE = {torch.float16: 0, torch.bfloat16: 1}


class PaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lock = threading.Lock()
_lib = None


def library(path: str | None = None):
    """The loaded libpa.so (ctypes), with argument types declared."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"{p} is not built; run `python -m paged_kv_cache_34_gb300.build` "
                "(there is no fallback implementation)")
        lib = ctypes.CDLL(p)
        c = ctypes
        V, I32, I64, F, SZ = c.c_void_p, c.c_int32, c.c_int64, c.c_float, c.c_size_t
        lib.pa_abi_version.argtypes, lib.pa_abi_version.restype = [], I32
        lib.pa_status_string.argtypes, lib.pa_status_string.restype = [c.c_int], c.c_char_p
        lib.pa_last_cuda_error.argtypes, lib.pa_last_cuda_error.restype = [], I32
        lib.pa_debug_set_wait_limit_ns.argtypes = [c.c_uint64]
        lib.pa_debug_set_wait_limit_ns.restype = None
        lib.pa_reshape_and_cache.argtypes = [V, V, I64, V, V, V, I32, I32, I32, I32, I64,
                                             c.c_int, V, V]
        lib.pa_reshape_and_cache.restype = c.c_int
        lib.pa_rope_and_cache.argtypes = [V, I64, V, I64, V, I64, V, V, I64, V, V, I64, I32, I32, V,
                                          V, F, V, V, V, I32, I32, I32, I32, I32, I64, c.c_int, V,
                                          V]
        lib.pa_rope_and_cache.restype = c.c_int
        lib.pa_decode_plan.argtypes = [I32, I32, I32, I32, I32, I32,
                                       c.POINTER(I32), c.POINTER(SZ)]
        lib.pa_decode_plan.restype = c.c_int
        lib.pa_decode.argtypes = [V, I64, V, I64, V, V, V, I64, I32, V, I32, I32, I32, I32,
                                  I32, I64, F, I32, I32, V, SZ, c.c_int, V, V]
        lib.pa_decode.restype = c.c_int
        lib.pa_decode_write.argtypes = [V, I64, V, I64, V, V, I64, V, V, V, I32, V, I64, I32,
                                        V, I32, I32, I32, I32, I32, I64, F, I32, I32, V, SZ,
                                        c.c_int, V, V]
        lib.pa_decode_write.restype = c.c_int
        lib.pa_prefill_varlen.argtypes = [V, I64, V, I64, V, V, V, I64, I32, V, V, I32, I32,
                                          I32, I32, I32, I32, I32, I32, I64, F, I32, c.c_int,
                                          V, V]
        lib.pa_prefill_varlen.restype = c.c_int
        lib.pa_reshape_and_cache_int8.argtypes = [V, V, I64, V, V, V, I32, I32, I32, I32, I64,
                                                  V, V, c.c_int, V, V]
        lib.pa_reshape_and_cache_int8.restype = c.c_int
        lib.pa_copy_blocks.argtypes = [V, V, I64, I64, V, I32, V, V]
        lib.pa_copy_blocks.restype = c.c_int
        lib.pa_build_tables.argtypes = [V, I64, I32, V, V, V, V, I32, V, V, V, V, V, I32, I32,
                                        I32, I64, V, V]
        lib.pa_build_tables.restype = c.c_int
        lib.pa_attention_varlen.argtypes = [V, I64, V, I64, V, V, I64, V, I32, I32, I32, I32,
                                            I32, I32, F, I32, c.c_int, V, V]
        lib.pa_attention_varlen.restype = c.c_int
        lib.pa_decode_shared_plan.argtypes = [I32] * 7 + [c.POINTER(SZ)]
        lib.pa_decode_shared_plan.restype = c.c_int
        lib.pa_decode_shared.argtypes = [V, I64, V, I64, V, V, V, I64, I32, V, V, V, I32, I32,
                                         I32, I32, I32, I32, I64, F, I32, I32, V, SZ, c.c_int,
                                         V, V]
        lib.pa_decode_shared.restype = c.c_int
        lib.pa_decode_int8.argtypes = [V, I64, V, I64, V, V, V, I64, I32, V, I32, I32, I32,
                                       I32, I32, I64, V, V, F, I32, I32, V, SZ, c.c_int, V, V]
        lib.pa_decode_int8.restype = c.c_int
        lib.pa_decode_write_int8.argtypes = [V, I64, V, I64, V, V, I64, V, V, V, I32, V, I64,
                                             I32, V, I32, I32, I32, I32, I32, I64, V, V, F, I32,
                                             I32, V, SZ, c.c_int, V, V]
        lib.pa_decode_write_int8.restype = c.c_int
        lib.pa_reshape_and_cache_fp8.argtypes = lib.pa_reshape_and_cache_int8.argtypes
        lib.pa_reshape_and_cache_fp8.restype = c.c_int
        lib.pa_decode_fp8.argtypes = lib.pa_decode_int8.argtypes
        lib.pa_decode_fp8.restype = c.c_int
        lib.pa_reshape_and_cache_fp4.argtypes = lib.pa_reshape_and_cache_int8.argtypes
        lib.pa_reshape_and_cache_fp4.restype = c.c_int
        lib.pa_gather_cache_fp4.argtypes = [V, I64, V, I64, I32, V, V, V, I64, I32, V, V, I32, I32,
                                            I32, I32, I32, I64, V, V, c.c_int, V, V]
        lib.pa_gather_cache_fp4.restype = c.c_int
        lib.pa_decode_fp4_plan.argtypes = [I32] * 5 + [c.POINTER(SZ)]
        lib.pa_decode_fp4_plan.restype = c.c_int
        lib.pa_decode_fp4.argtypes = [V, I64, V, I64, V, V, V, I64, I32, V, I32, I32, I32, I32, I32,
                                      I64, V, V, F, I32, V, SZ, c.c_int, V, V]
        lib.pa_decode_fp4.restype = c.c_int
        lib.pa_decode_write_fp4.argtypes = [V, I64, V, I64, V, V, I64, V, V, V, I32, V, I64, I32, V,
                                            I32, I32, I32, I32, I32, I64, V, V, F, I32, V, SZ,
                                            c.c_int, V, V]
        lib.pa_decode_write_fp4.restype = c.c_int
        lib.pa_decode_write_fp8.argtypes = lib.pa_decode_write_int8.argtypes
        lib.pa_decode_write_fp8.restype = c.c_int
        if path is None:
            _lib = lib
        return lib


def _check(lib, status: int, what: str):
    if status != 0:
        msg = lib.pa_status_string(status).decode()
        if status == 6:
            msg += f" (cudaError {lib.pa_last_cuda_error()})"
        raise PaError(status, f"{what}: {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _rows(t, name):
    """(row stride in elements) of a [rows, heads, head_dim] view with
    contiguous heads."""
    st = t.stride()
    if len(st) != 3 or st[2] != 1 or st[1] != t.shape[2]:
        raise ValueError(f"{name} must be [rows, heads, head_dim] with contiguous heads")
    return st[0]


def pa_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, *,
                         d_error=None, stream=None, lib=None):
    """key/value [N, Hkv, D] (equal row strides); caches [NB, bs, Hkv, D]
    contiguous; slot_mapping int64 [N]."""
    lib = lib or library()
    ks = _rows(key, "key")
    if _rows(value, "value") != ks:
        raise ValueError("key and value must share a row stride")
    if not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, D]")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    nb, bs, hkv, d = key_cache.shape
    st = lib.pa_reshape_and_cache(_ptr(key), _ptr(value), ks, _ptr(key_cache),
                                  _ptr(value_cache), _ptr(slot_mapping), key.shape[0], hkv, d,
                                  bs, nb, _DTYPE[key.dtype], _ptr(d_error), _stream(stream))
    _check(lib, st, "pa_reshape_and_cache")


def _row(t, d, name):
    """_rows of a tensor that is known to have three dimensions, the last d."""
    st = t.stride()
    if st[1] != d or st[2] != 1:
        raise ValueError(f"{name} must be [rows, heads, head_dim] with contiguous heads")
    return st[0]


def _rope(what, query_out, key_out, query, key, value, key_cache, value_cache, slot_mapping,
          positions, cos_sin, interleaved, q_weight, k_weight, eps, d_error, stream, lib):
    lib = lib or _lib or library()
    shape, kshape, dtype, dev = query.shape, key.shape, query.dtype, query.get_device()
    t, hq, d = shape
    tk, hkv, dk = kshape
    if query_out.shape != shape or tk != t or dk != d:
        raise ValueError("query_out/query must be [T, Hq, D] and key [T, Hkv, D]")
    if dtype not in _DTYPE or query_out.dtype is not dtype or key.dtype is not dtype:
        raise ValueError("query_out, query and key must share a dtype, float16 or bfloat16")
    if query_out.get_device() != dev or key.get_device() != dev:
        _bad_device("query_out or key", dev)
    ks = _row(key, d, "key")
    kos = ko = v = kc = vc = sm = pos = cs = qw = kw = None
    rot = most = bs = nb = 0
    if key_out is not None:
        if key_out.shape != kshape or key_out.dtype is not dtype:
            raise ValueError("key_out must be like key")
        if key_out.get_device() != dev:
            _bad_device("key_out", dev)
        kos, ko = _row(key_out, d, "key_out"), key_out.data_ptr()
    if key_cache is None or value_cache is None or slot_mapping is None:
        if not (key_cache is None and value_cache is None and slot_mapping is None):
            raise ValueError("caches and slot_mapping must be given together")
    else:
        if value is None:
            raise ValueError("value must be given with the caches")
        cshape = key_cache.shape
        nb, bs, hc, dc = cshape
        if value.shape != kshape or value.dtype is not dtype or _row(value, d, "value") != ks:
            raise ValueError("value must be like key, with its row stride")
        if hc != hkv or dc != d or value_cache.shape != cshape \
                or key_cache.dtype is not dtype or value_cache.dtype is not dtype \
                or not key_cache.is_contiguous() or not value_cache.is_contiguous():
            raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, D] of key's "
                             "dtype")
        if not (value.get_device() == dev and key_cache.get_device() == dev
                and value_cache.get_device() == dev):
            _bad_device("value or caches", dev)
        if slot_mapping.dtype is not torch.int64 or slot_mapping.numel() != t \
                or slot_mapping.get_device() != dev or not slot_mapping.is_contiguous():
            _bad_vector(slot_mapping, t, torch.int64, "slot_mapping", dev)
        v, kc, vc = value.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr()
        sm = slot_mapping.data_ptr()
    if cos_sin is not None:
        if positions is None:
            raise ValueError("positions must be given with cos_sin")
        if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous float32 tensor [max_position, rot_dim]")
        if cos_sin.get_device() != dev:
            _bad_device("cos_sin", dev)
        if positions.dtype is not torch.int32 or positions.numel() != t \
                or positions.get_device() != dev or not positions.is_contiguous():
            _bad_vector(positions, t, torch.int32, "positions", dev)
        most, rot = cos_sin.shape
        pos, cs = positions.data_ptr(), cos_sin.data_ptr()
    if q_weight is not None:
        qw = _weight(q_weight, d, dtype, "q_weight", dev)
    if k_weight is not None:
        kw = _weight(k_weight, d, dtype, "k_weight", dev)
    if d_error is not None:
        _check_error(d_error, dev)
        d_error = d_error.data_ptr()
    _current(dev)
    st = lib.pa_rope_and_cache(
        query_out.data_ptr(), _row(query_out, d, "query_out"), ko, kos or 0, query.data_ptr(),
        _row(query, d, "query"), key.data_ptr(), v, ks, pos, cs, most, rot,
        1 if interleaved else 0, qw, kw, eps, kc, vc, sm, t, hq, hkv, d, bs, nb, _DTYPE[dtype],
        d_error, _raw_stream(stream, dev))
    if st:
        _check(lib, st, what)


def _weight(w, d, dtype, name, dev):
    if w.dtype is not dtype or w.numel() != d or not w.is_contiguous() or w.get_device() != dev:
        _bad_vector(w, d, dtype, name, dev)
    return w.data_ptr()


def pa_rope_and_cache(query_out, query, key, value, key_cache, value_cache, slot_mapping, positions,
                      cos_sin, *, key_out=None, interleaved=False, q_weight=None, k_weight=None,
                      eps=1e-6, d_error=None, stream=None, lib=None):
    """Norms (where weights [D] are given) and rotation of a step's query and
    key heads, and its cache write, in one pass: query_out/query [T, Hq, D],
    key/value [T, Hkv, D] (equal row strides), caches [NB, bs, Hkv, D],
    slot_mapping int64 [T] (negative: no cache write), positions int32 [T],
    cos_sin float32 [max_position, rot_dim] (cosines, then sines; None: no
    rotation).  The pairs rotated are (i, i + rot_dim/2), or (2i, 2i + 1) when
    ``interleaved``.  ``key_out`` also takes the key rows; query_out and
    key_out may be query and key themselves."""
    _rope("pa_rope_and_cache", query_out, key_out, query, key, value, key_cache, value_cache,
          slot_mapping, positions, cos_sin, interleaved, q_weight, k_weight, eps, d_error, stream,
          lib)


def pa_qk_norm_rope(query_out, key_out, query, key, positions, cos_sin, *, interleaved=False,
                    q_weight=None, k_weight=None, eps=1e-6, d_error=None, stream=None, lib=None):
    """pa_rope_and_cache without a cache: norms and rotation of the query and
    key heads into query_out [T, Hq, D] and key_out [T, Hkv, D] (query and key
    themselves, for example)."""
    _rope("pa_qk_norm_rope", query_out, key_out, query, key, None, None, None, None, positions,
          cos_sin, interleaved, q_weight, k_weight, eps, d_error, stream, lib)


def _scales(t, hkv, what):
    if t.dtype != torch.float32 or t.numel() != hkv or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor of num_kv_heads values")
    return _ptr(t)


_POOL8 = {"int8": (torch.int8,), "fp8": (torch.uint8, torch.float8_e4m3fn)}


def _check_pools8(fmt, key_cache, value_cache):
    if key_cache.dtype not in _POOL8[fmt] or value_cache.dtype not in _POOL8[fmt]:
        names = " or ".join(str(t).replace("torch.", "") for t in _POOL8[fmt])
        raise ValueError(f"{fmt.upper()} caches must be {names}")
    if not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, D]")


def _write8(fmt, key, value, key_cache, value_cache, slot_mapping, k_scale, v_scale, d_error,
            stream, lib):
    lib = lib or library()
    ks = _rows(key, "key")
    if _rows(value, "value") != ks:
        raise ValueError("key and value must share a row stride")
    _check_pools8(fmt, key_cache, value_cache)
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    nb, bs, hkv, d = key_cache.shape
    name = f"pa_reshape_and_cache_{fmt}"
    st = getattr(lib, name)(
        _ptr(key), _ptr(value), ks, _ptr(key_cache), _ptr(value_cache), _ptr(slot_mapping),
        key.shape[0], hkv, d, bs, nb, _scales(k_scale, hkv, "k_scale"),
        _scales(v_scale, hkv, "v_scale"), _DTYPE[key.dtype], _ptr(d_error), _stream(stream))
    _check(lib, st, name)


def pa_reshape_and_cache_int8(key, value, key_cache, value_cache, slot_mapping, k_scale,
                              v_scale, *, d_error=None, stream=None, lib=None):
    """pa_reshape_and_cache into INT8 pools: caches int8 [NB, bs, Hkv, D];
    k_scale / v_scale float32 [Hkv] (per-KV-head dequantisation scales)."""
    _write8("int8", key, value, key_cache, value_cache, slot_mapping, k_scale, v_scale,
            d_error, stream, lib)


def pa_reshape_and_cache_fp8(key, value, key_cache, value_cache, slot_mapping, k_scale,
                             v_scale, *, d_error=None, stream=None, lib=None):
    """pa_reshape_and_cache into FP8 pools: caches of E4M3 codes (uint8 or
    float8_e4m3fn) [NB, bs, Hkv, D]; k_scale / v_scale float32 [Hkv]."""
    _write8("fp8", key, value, key_cache, value_cache, slot_mapping, k_scale, v_scale,
            d_error, stream, lib)


def _pools4(key_cache, value_cache, dev):
    """(num_blocks, num_kv_heads, block_size, head_dim) of a pair of FP4 pools."""
    shape = key_cache.shape
    if key_cache.dtype is not torch.uint8 or value_cache.dtype is not torch.uint8 \
            or len(shape) != 4 or value_cache.shape != shape or shape[3] % 9 \
            or not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError("FP4 caches must be contiguous uint8 [num_blocks, Hkv, block_size / 8, "
                         "9 * head_dim / 2]")
    if key_cache.get_device() != dev or value_cache.get_device() != dev:
        _bad_device("caches", dev)
    nb, hkv, tiles, width = shape
    return nb, hkv, 8 * tiles, width // 9 * 2


def _scales4(k, v, hkv, dev):
    f32 = torch.float32
    if not (k.dtype is f32 and v.dtype is f32 and k.numel() == hkv and v.numel() == hkv
            and k.is_contiguous() and v.is_contiguous() and k.get_device() == dev
            and v.get_device() == dev):
        for t, what in ((k, "k_scale"), (v, "v_scale")):
            if t.dtype is not f32 or t.numel() != hkv or not t.is_contiguous() \
                    or t.get_device() != dev:
                _bad_vector(t, hkv, f32, what, dev)
    return k.data_ptr(), v.data_ptr()


def _new_rows4(key, value, slot_mapping, hkv, d, dev):
    """(row stride, token count) of the rows that a write into FP4 pools takes."""
    shape, dtype = key.shape, key.dtype
    n, h, dk = shape
    if dtype not in _DTYPE or value.dtype is not dtype or value.shape != shape or h != hkv or dk != d:
        raise ValueError("key and value must be [N, Hkv, D] of one dtype, float16 or bfloat16")
    ks = _row(key, d, "key")
    if _row(value, d, "value") != ks:
        raise ValueError("key and value must share a row stride")
    if key.get_device() != dev or value.get_device() != dev:
        _bad_device("key or value", dev)
    if slot_mapping.dtype is not torch.int64 or slot_mapping.numel() != n \
            or slot_mapping.get_device() != dev or not slot_mapping.is_contiguous():
        _bad_vector(slot_mapping, n, torch.int64, "slot_mapping", dev)
    return ks, n


def pa_reshape_and_cache_fp4(key, value, key_cache, value_cache, slot_mapping, k_scale, v_scale,
                             *, d_error=None, stream=None, lib=None):
    """pa_reshape_and_cache into FP4 pools: caches uint8 [NB, Hkv, bs / 8, 9 D / 2]
    (tiles of eight tokens: E2M1 codes, then E4M3 group scales); k_scale / v_scale
    float32 [Hkv], between 2**-64 and 2**64 (absmax / 2688, for example)."""
    lib = lib or _lib or library()
    dev = key.get_device()
    nb, hkv, bs, d = _pools4(key_cache, value_cache, dev)
    ks, n = _new_rows4(key, value, slot_mapping, hkv, d, dev)
    k_sc, v_sc = _scales4(k_scale, v_scale, hkv, dev)
    if d_error is not None:
        _check_error(d_error, dev)
    _current(dev)
    st = lib.pa_reshape_and_cache_fp4(
        key.data_ptr(), value.data_ptr(), ks, key_cache.data_ptr(), value_cache.data_ptr(),
        slot_mapping.data_ptr(), n, hkv, d, bs, nb, k_sc, v_sc, _DTYPE[key.dtype],
        None if d_error is None else d_error.data_ptr(), _raw_stream(stream, dev))
    if st:
        _check(lib, st, "pa_reshape_and_cache_fp4")


def _table4(block_table, s, dev):
    """(row stride, width) of a block table int32 [s, max_blocks]."""
    if block_table.dtype is not torch.int32 or block_table.dim() != 2 or block_table.shape[0] != s:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks]")
    stride, inner = block_table.stride()
    width = block_table.shape[1]
    if width > 1 and inner != 1:
        raise ValueError("block_table must have contiguous rows")
    if block_table.get_device() != dev:
        _bad_device("block_table", dev)
    return (stride if s > 1 else width), width


def pa_gather_cache_fp4(key_out, value_out, key_cache, value_cache, block_table, context_lens,
                        row_starts, k_scale, v_scale, *, max_context_len, d_error=None, stream=None,
                        lib=None):
    """The rows that FP4 pools hold, in 16 bits: position j < context_lens[b] of
    sequence b goes to row row_starts[b] + j (both int32 [S]) of key_out and
    value_out [R, Hkv, D]; other rows are left as they were."""
    lib = lib or _lib or library()
    dev, s = key_out.get_device(), context_lens.numel()
    nb, hkv, bs, d = _pools4(key_cache, value_cache, dev)
    r = key_out.shape[0]
    if key_out.dtype not in _DTYPE or value_out.dtype is not key_out.dtype \
            or key_out.shape != (r, hkv, d) or value_out.shape != (r, hkv, d):
        raise ValueError("key_out and value_out must be [R, Hkv, D] of one dtype, float16 or "
                         "bfloat16")
    if value_out.get_device() != dev:
        _bad_device("value_out", dev)
    ks, vs = _row(key_out, d, "key_out"), _row(value_out, d, "value_out")
    stride, width = _table4(block_table, s, dev)
    for t, name in ((context_lens, "context_lens"), (row_starts, "row_starts")):
        if t.dtype is not torch.int32 or t.numel() != s or t.get_device() != dev \
                or not t.is_contiguous():
            _bad_vector(t, s, torch.int32, name, dev)
    k_sc, v_sc = _scales4(k_scale, v_scale, hkv, dev)
    max_context_len = _bound(max_context_len, "max_context_len")
    if d_error is not None:
        _check_error(d_error, dev)
    _current(dev)
    st = lib.pa_gather_cache_fp4(
        key_out.data_ptr(), ks, value_out.data_ptr(), vs, r, key_cache.data_ptr(),
        value_cache.data_ptr(), block_table.data_ptr(), stride, width, context_lens.data_ptr(),
        row_starts.data_ptr(), s, max_context_len, hkv, d, bs, nb, k_sc, v_sc,
        _DTYPE[key_out.dtype], None if d_error is None else d_error.data_ptr(),
        _raw_stream(stream, dev))
    if st:
        _check(lib, st, "pa_gather_cache_fp4")


def pa_copy_blocks(key_cache, value_cache, block_mapping, *, d_error=None, stream=None,
                   lib=None):
    """Copy-on-write of whole blocks: for each row (src, dst) of block_mapping
    (int64 [n, 2] on the device), block dst of both pools receives block src.
    The pools are contiguous [num_blocks, ...] tensors of one shape and dtype
    (16-bit or INT8 pools alike)."""
    lib = lib or library()
    if key_cache.shape != value_cache.shape or key_cache.dtype != value_cache.dtype:
        raise ValueError("key_cache and value_cache must share shape and dtype")
    if not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, ...]")
    if block_mapping.dtype != torch.int64 or not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be a contiguous int64 tensor [n, 2]")
    if block_mapping.numel() % 2:
        raise ValueError("block_mapping must hold (src, dst) pairs")
    nb = key_cache.shape[0]
    block_bytes = key_cache.element_size()
    for n in key_cache.shape[1:]:
        block_bytes *= n
    st = lib.pa_copy_blocks(_ptr(key_cache), _ptr(value_cache), block_bytes, nb,
                            _ptr(block_mapping), block_mapping.numel() // 2, _ptr(d_error),
                            _stream(stream))
    _check(lib, st, "pa_copy_blocks")


def _bad_vector(t, n, dtype, name, dev):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values".replace(
            "torch.", ""))
    _bad_device(name, dev)


def _bad_device(name, dev):
    raise ValueError(f"{name} is not on the CUDA device of the call ({dev}): a pointer of another "
                     "device, or of the host, would fault")


def _check_error(t, dev):
    if t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError("d_error must be an int32 tensor")
    if t.get_device() != dev:
        _bad_device("d_error", dev)


def _current(dev):
    """The call's device is the current one, where its kernels are launched."""
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("the tensors must be on the current CUDA device")


def _bound(v, name):
    """A host bound as the C int32 it is passed as (ctypes would wrap a larger
    one: 2**32 to 0, nothing to do)."""
    v = int(v)
    if not 0 <= v <= 0x7fffffff:
        raise ValueError(f"{name} must be between 0 and 2**31 - 1")
    return v


def _raw_stream(stream, dev):
    """The cudaStream_t of `stream`, or of the current stream (without building
    a stream object, which takes 3 us)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def pa_build_tables(block_table, context_lens, query_lens, free_blocks, num_free,
                    context_lens_out, cu_seqlens_q, slot_mapping, num_free_out, *, block_size,
                    num_blocks, positions=None, d_error=None, stream=None, lib=None):
    """A serving step's metadata from request lengths: request b holds
    context_lens[b] cached tokens and gets query_lens[b] new ones (int32 [S]).
    Writes context_lens_out int32 [S], cu_seqlens_q int32 [S+1], slot_mapping
    int64 [T] and positions int32 [T] (entries past the step's tokens get -1
    and 0), the block_table (int32 [S, max_blocks]) entries of the blocks
    taken off the end of free_blocks[:num_free], and num_free_out int32 [1].
    No output may overlap an input."""
    lib = lib or _lib or library()
    s, t, nfree = context_lens.shape[0], slot_mapping.shape[0], free_blocks.shape[0]
    i32, dev = torch.int32, context_lens.get_device()
    if block_table.dtype is not i32 or block_table.dim() != 2 or block_table.shape[0] != s:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks]")
    stride, inner = block_table.stride()
    width = block_table.shape[1]
    if width > 1 and inner != 1:
        raise ValueError("block_table must have contiguous rows")
    # one expression for what a right call passes (a loop over the tensors takes
    # 1.4 us longer, and the host's time is this call's); which is wrong, below
    pos_ok = positions is None or (positions.dtype is i32 and positions.numel() == t
                                   and positions.get_device() == dev
                                   and positions.is_contiguous())
    if not (pos_ok and context_lens.dtype is i32 and query_lens.dtype is i32
            and free_blocks.dtype is i32 and num_free.dtype is i32
            and context_lens_out.dtype is i32 and cu_seqlens_q.dtype is i32
            and num_free_out.dtype is i32 and slot_mapping.dtype is torch.int64
            and context_lens.numel() == s and query_lens.numel() == s
            and free_blocks.numel() == nfree and num_free.numel() == 1
            and context_lens_out.numel() == s and cu_seqlens_q.numel() == s + 1
            and num_free_out.numel() == 1 and slot_mapping.numel() == t
            and query_lens.get_device() == dev and free_blocks.get_device() == dev
            and num_free.get_device() == dev and context_lens_out.get_device() == dev
            and cu_seqlens_q.get_device() == dev and num_free_out.get_device() == dev
            and slot_mapping.get_device() == dev and context_lens.is_contiguous()
            and query_lens.is_contiguous() and free_blocks.is_contiguous()
            and context_lens_out.is_contiguous() and cu_seqlens_q.is_contiguous()
            and slot_mapping.is_contiguous()):
        vectors = [(context_lens, s, i32, "context_lens"), (query_lens, s, i32, "query_lens"),
                   (free_blocks, nfree, i32, "free_blocks"), (num_free, 1, i32, "num_free"),
                   (context_lens_out, s, i32, "context_lens_out"),
                   (cu_seqlens_q, s + 1, i32, "cu_seqlens_q"),
                   (slot_mapping, t, torch.int64, "slot_mapping"),
                   (num_free_out, 1, i32, "num_free_out")]
        if positions is not None:
            vectors.append((positions, t, i32, "positions"))
        for v in vectors:
            if v[0].dtype is not v[2] or v[0].numel() != v[1] or v[0].get_device() != dev \
                    or not v[0].is_contiguous():
                _bad_vector(*v, dev)
    if block_table.get_device() != dev:
        _bad_device("block_table", dev)
    if d_error is not None:
        _check_error(d_error, dev)
    _current(dev)
    st = lib.pa_build_tables(block_table.data_ptr(), stride if s > 1 else width, width,
                             context_lens.data_ptr(), query_lens.data_ptr(),
                             free_blocks.data_ptr(), num_free.data_ptr(), nfree,
                             context_lens_out.data_ptr(), cu_seqlens_q.data_ptr(),
                             slot_mapping.data_ptr(),
                             None if positions is None else positions.data_ptr(),
                             num_free_out.data_ptr(), s, t, block_size, num_blocks,
                             None if d_error is None else d_error.data_ptr(),
                             _raw_stream(stream, dev))
    if st:
        _check(lib, st, "pa_build_tables")


def pa_debug_set_wait_limit_ns(ns: int, *, lib=None):
    """Bound (ns) of the kernels' pipeline waits for later launches; 0 = the
    default 2 s.  A testing aid: lets a test make waits run out."""
    (lib or library()).pa_debug_set_wait_limit_ns(int(ns))


def pa_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                   partition_size=0, lib=None):
    """(partition_size, workspace_bytes) that pa_decode will use."""
    lib = lib or library()
    p = ctypes.c_int32(0)
    ws = ctypes.c_size_t(0)
    st = lib.pa_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                            partition_size, ctypes.byref(p), ctypes.byref(ws))
    _check(lib, st, "pa_decode_plan")
    return p.value, ws.value


def pa_decode(out, query, key_cache, value_cache, block_table, context_lens, *, scale,
              max_context_len, partition_size=0, workspace=None, d_error=None, stream=None,
              lib=None):
    """out/query [S, Hq, D]; caches [NB, bs, Hkv, D]; block_table int32
    [S, max_blocks]; context_lens int32 [S].  ``max_context_len`` is the
    host-side upper bound of context_lens.  A workspace is allocated with
    torch when the plan needs one and none is given."""
    lib = lib or library()
    s, hq, d = query.shape
    nb, bs, hkv, _ = key_cache.shape
    P, need = pa_decode_plan(s, hq, hkv, d, max_context_len, partition_size, lib=lib)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_table and context_lens must be int32")
    st = lib.pa_decode(_ptr(out), _rows(out, "out"), _ptr(query), _rows(query, "query"),
                       _ptr(key_cache), _ptr(value_cache), _ptr(block_table),
                       block_table.stride(0), block_table.shape[1], _ptr(context_lens), s, hq,
                       hkv, d, bs, nb, float(scale), int(max_context_len), P,
                       _ptr(workspace), wbytes, _DTYPE[query.dtype], _ptr(d_error),
                       _stream(stream))
    _check(lib, st, "pa_decode")
    return out


def _decode8(fmt, out, query, key_cache, value_cache, block_table, context_lens, k_scale,
             v_scale, scale, max_context_len, partition_size, workspace, d_error, stream, lib):
    lib = lib or library()
    s, hq, d = query.shape
    nb, bs, hkv, _ = key_cache.shape
    _check_pools8(fmt, key_cache, value_cache)
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_table and context_lens must be int32")
    P, need = pa_decode_plan(s, hq, hkv, d, max_context_len, partition_size, lib=lib)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    name = f"pa_decode_{fmt}"
    st = getattr(lib, name)(
        _ptr(out), _rows(out, "out"), _ptr(query), _rows(query, "query"), _ptr(key_cache),
        _ptr(value_cache), _ptr(block_table), block_table.stride(0), block_table.shape[1],
        _ptr(context_lens), s, hq, hkv, d, bs, nb, _scales(k_scale, hkv, "k_scale"),
        _scales(v_scale, hkv, "v_scale"), float(scale), int(max_context_len), P,
        _ptr(workspace), wbytes, _DTYPE[query.dtype], _ptr(d_error), _stream(stream))
    _check(lib, st, name)
    return out


def pa_decode_int8(out, query, key_cache, value_cache, block_table, context_lens, k_scale,
                   v_scale, *, scale, max_context_len, partition_size=0, workspace=None,
                   d_error=None, stream=None, lib=None):
    """pa_decode over INT8 pools (int8 [NB, bs, Hkv, D], head_dim 64 or 128) with
    per-KV-head float32 scales k_scale / v_scale [Hkv]."""
    return _decode8("int8", out, query, key_cache, value_cache, block_table, context_lens,
                    k_scale, v_scale, scale, max_context_len, partition_size, workspace,
                    d_error, stream, lib)


def pa_decode_fp8(out, query, key_cache, value_cache, block_table, context_lens, k_scale,
                  v_scale, *, scale, max_context_len, partition_size=0, workspace=None,
                  d_error=None, stream=None, lib=None):
    """pa_decode over FP8 pools (E4M3 codes, uint8 or float8_e4m3fn
    [NB, bs, Hkv, D], head_dim 64 or 128) with per-KV-head float32 scales."""
    return _decode8("fp8", out, query, key_cache, value_cache, block_table, context_lens,
                    k_scale, v_scale, scale, max_context_len, partition_size, workspace,
                    d_error, stream, lib)


def pa_decode_write(out, query, key, value, key_cache, value_cache, slot_mapping, block_table,
                    context_lens, *, scale, max_context_len, partition_size=0, workspace=None,
                    d_error=None, stream=None, lib=None):
    """One decode step in one call: pa_reshape_and_cache(key, value, ...,
    slot_mapping) then pa_decode(...), the decode overlapping the write.
    Arguments as for those two functions."""
    lib = lib or library()
    s, hq, d = query.shape
    nb, bs, hkv, _ = key_cache.shape
    ks = _rows(key, "key")
    if _rows(value, "value") != ks:
        raise ValueError("key and value must share a row stride")
    if not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, D]")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_table and context_lens must be int32")
    P, need = pa_decode_plan(s, hq, hkv, d, max_context_len, partition_size, lib=lib)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.pa_decode_write(_ptr(out), _rows(out, "out"), _ptr(query), _rows(query, "query"),
                             _ptr(key), _ptr(value), ks, _ptr(key_cache), _ptr(value_cache),
                             _ptr(slot_mapping), key.shape[0], _ptr(block_table),
                             block_table.stride(0), block_table.shape[1], _ptr(context_lens), s,
                             hq, hkv, d, bs, nb, float(scale), int(max_context_len), P,
                             _ptr(workspace), wbytes, _DTYPE[query.dtype], _ptr(d_error),
                             _stream(stream))
    _check(lib, st, "pa_decode_write")
    return out


def _decode_write8(fmt, out, query, key, value, key_cache, value_cache, slot_mapping,
                   block_table, context_lens, k_scale, v_scale, scale, max_context_len,
                   partition_size, workspace, d_error, stream, lib):
    lib = lib or library()
    s, hq, d = query.shape
    nb, bs, hkv, _ = key_cache.shape
    ks = _rows(key, "key")
    if _rows(value, "value") != ks:
        raise ValueError("key and value must share a row stride")
    _check_pools8(fmt, key_cache, value_cache)
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_table and context_lens must be int32")
    P, need = pa_decode_plan(s, hq, hkv, d, max_context_len, partition_size, lib=lib)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    name = f"pa_decode_write_{fmt}"
    st = getattr(lib, name)(
        _ptr(out), _rows(out, "out"), _ptr(query), _rows(query, "query"), _ptr(key),
        _ptr(value), ks, _ptr(key_cache), _ptr(value_cache), _ptr(slot_mapping), key.shape[0],
        _ptr(block_table), block_table.stride(0), block_table.shape[1], _ptr(context_lens), s,
        hq, hkv, d, bs, nb, _scales(k_scale, hkv, "k_scale"), _scales(v_scale, hkv, "v_scale"),
        float(scale), int(max_context_len), P, _ptr(workspace), wbytes, _DTYPE[query.dtype],
        _ptr(d_error), _stream(stream))
    _check(lib, st, name)
    return out


def pa_decode_write_int8(out, query, key, value, key_cache, value_cache, slot_mapping,
                         block_table, context_lens, k_scale, v_scale, *, scale, max_context_len,
                         partition_size=0, workspace=None, d_error=None, stream=None, lib=None):
    """One decode step over INT8 pools in one call: pa_reshape_and_cache_int8
    then pa_decode_int8, the decode overlapping the write.  Arguments as for
    those two functions."""
    return _decode_write8("int8", out, query, key, value, key_cache, value_cache, slot_mapping,
                          block_table, context_lens, k_scale, v_scale, scale, max_context_len,
                          partition_size, workspace, d_error, stream, lib)


def pa_decode_write_fp8(out, query, key, value, key_cache, value_cache, slot_mapping,
                        block_table, context_lens, k_scale, v_scale, *, scale, max_context_len,
                        partition_size=0, workspace=None, d_error=None, stream=None, lib=None):
    """One decode step over FP8 pools in one call: pa_reshape_and_cache_fp8
    then pa_decode_fp8.  Arguments as for those two functions."""
    return _decode_write8("fp8", out, query, key, value, key_cache, value_cache, slot_mapping,
                          block_table, context_lens, k_scale, v_scale, scale, max_context_len,
                          partition_size, workspace, d_error, stream, lib)


def pa_decode_fp4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len, lib=None):
    """The workspace bytes pa_decode_fp4 needs for this shape."""
    lib = lib or _lib or library()
    ws = ctypes.c_size_t(0)
    st = lib.pa_decode_fp4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                _bound(max_context_len, "max_context_len"), ctypes.byref(ws))
    if st:
        _check(lib, st, "pa_decode_fp4_plan")
    return ws.value


def _decode4(what, out, query, new, key_cache, value_cache, block_table, context_lens, k_scale,
             v_scale, scale, max_context_len, workspace, d_error, stream, lib):
    lib = lib or _lib or library()
    s, hq, dq = query.shape
    dtype, dev = query.dtype, query.get_device()
    nb, hkv, bs, d = _pools4(key_cache, value_cache, dev)
    if out.shape != query.shape or dq != d or dtype not in _DTYPE or out.dtype is not dtype:
        raise ValueError("out/query must be [S, Hq, D] of one dtype, float16 or bfloat16")
    os, qs = _row(out, d, "out"), _row(query, d, "query")
    stride, width = _table4(block_table, s, dev)
    if context_lens.dtype is not torch.int32 or context_lens.numel() != s \
            or context_lens.get_device() != dev or not context_lens.is_contiguous():
        _bad_vector(context_lens, s, torch.int32, "context_lens", dev)
    k_sc, v_sc = _scales4(k_scale, v_scale, hkv, dev)
    if out.get_device() != dev or workspace is not None and workspace.get_device() != dev:
        _bad_device("out or workspace", dev)
    max_context_len = _bound(max_context_len, "max_context_len")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    rows = ()
    if new is not None:
        key, value, slot_mapping = new
        ks, n = _new_rows4(key, value, slot_mapping, hkv, d, dev)
        if key.dtype is not dtype:
            raise ValueError("key and value must share query's dtype")
        rows = (key.data_ptr(), value.data_ptr(), ks, key_cache.data_ptr(), value_cache.data_ptr(),
                slot_mapping.data_ptr(), n)
    if d_error is not None:
        _check_error(d_error, dev)
    _current(dev)
    if workspace is None:
        need = pa_decode_fp4_plan(s, hq, hkv, d, max_context_len, lib=lib)
        # on the call's stream: a later allocation of another one must not get it
        with torch.cuda.stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    st = getattr(lib, what)(
        out.data_ptr(), os, query.data_ptr(), qs,
        *(rows or (key_cache.data_ptr(), value_cache.data_ptr())), block_table.data_ptr(), stride,
        width, context_lens.data_ptr(), s, hq, hkv, d, bs, nb, k_sc, v_sc, scale, max_context_len,
        workspace.data_ptr(), workspace.nbytes, _DTYPE[dtype],
        None if d_error is None else d_error.data_ptr(), _raw_stream(stream, dev))
    if st:
        _check(lib, st, what)
    return out


def pa_decode_fp4(out, query, key_cache, value_cache, block_table, context_lens, k_scale, v_scale,
                  *, scale, max_context_len, workspace=None, d_error=None, stream=None, lib=None):
    """pa_decode over FP4 pools (see pa_reshape_and_cache_fp4) with per-KV-head
    float32 scales.  A workspace is allocated with torch when none is given."""
    return _decode4("pa_decode_fp4", out, query, None, key_cache, value_cache, block_table,
                    context_lens, k_scale, v_scale, scale, max_context_len, workspace, d_error,
                    stream, lib)


def pa_decode_write_fp4(out, query, key, value, key_cache, value_cache, slot_mapping, block_table,
                        context_lens, k_scale, v_scale, *, scale, max_context_len, workspace=None,
                        d_error=None, stream=None, lib=None):
    """One decode step over FP4 pools in one call: pa_reshape_and_cache_fp4, then
    pa_decode_fp4.  Arguments as for those two functions."""
    return _decode4("pa_decode_write_fp4", out, query, (key, value, slot_mapping), key_cache,
                    value_cache, block_table, context_lens, k_scale, v_scale, scale,
                    max_context_len, workspace, d_error, stream, lib)


def pa_prefill_varlen(out, query, key_cache, value_cache, block_table, cu_seqlens_q,
                      context_lens, *, scale, max_seqlen_q, max_context_len, causal=True,
                      d_error=None, stream=None, lib=None):
    """out/query [T, Hq, D] packed by cu_seqlens_q int32 [S+1];
    context_lens int32 [S].  ``max_seqlen_q`` / ``max_context_len`` are host
    upper bounds; T (total_q) is taken from query.shape[0]."""
    lib = lib or library()
    t, hq, d = query.shape
    nb, bs, hkv, _ = key_cache.shape
    s = context_lens.shape[0]
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32 \
            or cu_seqlens_q.dtype != torch.int32:
        raise ValueError("block_table, cu_seqlens_q and context_lens must be int32")
    st = lib.pa_prefill_varlen(_ptr(out), _rows(out, "out"), _ptr(query), _rows(query, "query"),
                               _ptr(key_cache), _ptr(value_cache), _ptr(block_table),
                               block_table.stride(0), block_table.shape[1], _ptr(cu_seqlens_q),
                               _ptr(context_lens), s, t, int(max_seqlen_q),
                               int(max_context_len), hq, hkv, d, bs, nb, float(scale),
                               1 if causal else 0, _DTYPE[query.dtype], _ptr(d_error),
                               _stream(stream))
    _check(lib, st, "pa_prefill_varlen")
    return out


def pa_attention_varlen(out, query, key, value, cu_seqlens, *, scale, max_seqlen, causal=True,
                        d_error=None, stream=None, lib=None):
    """Attention of prompts packed one behind the other, over their own rows:
    out/query [T, Hq, D], key/value [T, Hkv, D] (equal row strides, e.g. views
    into one QKV buffer), cu_seqlens int32 [S+1].  ``max_seqlen`` is the host
    upper bound of the lengths (0: nothing to do); rows past cu_seqlens[S] are
    left alone."""
    lib = lib or _lib or library()
    t, hq, d = query.shape
    shape, dtype, n, dev = key.shape, query.dtype, cu_seqlens.numel(), query.get_device()
    if out.shape != query.shape or shape != value.shape or shape[0] != t or shape[2] != d:
        raise ValueError("out/query must be [T, Hq, D] and key/value [T, Hkv, D]")
    if dtype not in _DTYPE or out.dtype is not dtype or key.dtype is not dtype \
            or value.dtype is not dtype:
        raise ValueError("out, query, key and value must share a dtype, float16 or bfloat16")
    os, qs, ks = _rows(out, "out"), _rows(query, "query"), _rows(key, "key")
    if _rows(value, "value") != ks:
        raise ValueError("key and value must share a row stride")
    if cu_seqlens.dtype is not torch.int32 or n < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of num_seqs + 1 values")
    if not (out.get_device() == dev and key.get_device() == dev and value.get_device() == dev
            and cu_seqlens.get_device() == dev):
        _bad_device("out, key, value or cu_seqlens", dev)
    max_seqlen = _bound(max_seqlen, "max_seqlen")
    if d_error is not None:
        _check_error(d_error, dev)
    _current(dev)
    st = lib.pa_attention_varlen(out.data_ptr(), os, query.data_ptr(), qs, key.data_ptr(),
                                 value.data_ptr(), ks, cu_seqlens.data_ptr(), n - 1, t,
                                 max_seqlen, hq, shape[1], d, float(scale),
                                 1 if causal else 0, _DTYPE[dtype],
                                 None if d_error is None else d_error.data_ptr(),
                                 _raw_stream(stream, dev))
    if st:
        _check(lib, st, "pa_attention_varlen")
    return out


def pa_decode_shared_plan(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim,
                          max_context_len, max_prefix_len, lib=None):
    """The workspace bytes pa_decode_shared needs for this shape."""
    lib = lib or library()
    ws = ctypes.c_size_t(0)
    st = lib.pa_decode_shared_plan(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim,
                                   _bound(max_context_len, "max_context_len"),
                                   _bound(max_prefix_len, "max_prefix_len"), ctypes.byref(ws))
    _check(lib, st, "pa_decode_shared_plan")
    return ws.value


def pa_decode_shared(out, query, key_cache, value_cache, block_table, context_lens, group_starts,
                     prefix_lens, *, scale, max_context_len, max_prefix_len, workspace=None,
                     d_error=None, stream=None, lib=None):
    """pa_decode for a batch whose groups share a prefix: group g is sequences
    group_starts[g] .. group_starts[g+1]-1 (int32 [G+1]); the first
    prefix_lens[g] (int32 [G]) tokens of each are those of its first sequence's
    block_table row and are read once for the group.  ``max_context_len`` and
    ``max_prefix_len`` are host upper bounds.  A workspace is allocated with
    torch when none is given."""
    lib = lib or _lib or library()
    s, hq, d = query.shape
    nb, bs, hkv, dk = key_cache.shape
    g, dtype, i32, dev = prefix_lens.shape[0], query.dtype, torch.int32, query.get_device()
    if out.shape != query.shape or dk != d or value_cache.shape != key_cache.shape:
        raise ValueError("out/query must be [S, Hq, D], the caches [NB, bs, Hkv, D]")
    if dtype not in _DTYPE or out.dtype is not dtype or key_cache.dtype is not dtype \
            or value_cache.dtype is not dtype:
        raise ValueError("out, query and caches must share a dtype, float16 or bfloat16")
    if not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, D]")
    if block_table.dtype is not i32 or block_table.dim() != 2 or block_table.shape[0] != s:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks]")
    stride, inner = block_table.stride()
    width = block_table.shape[1]
    if width > 1 and inner != 1:
        raise ValueError("block_table must have contiguous rows")
    if not (context_lens.dtype is i32 and group_starts.dtype is i32 and prefix_lens.dtype is i32
            and context_lens.numel() == s and group_starts.numel() == g + 1
            and prefix_lens.numel() == g and context_lens.get_device() == dev
            and group_starts.get_device() == dev and prefix_lens.get_device() == dev
            and context_lens.is_contiguous() and group_starts.is_contiguous()
            and prefix_lens.is_contiguous()):
        for v in ((context_lens, s, i32, "context_lens"),
                  (group_starts, g + 1, i32, "group_starts"), (prefix_lens, g, i32, "prefix_lens")):
            if v[0].dtype is not i32 or v[0].numel() != v[1] or v[0].get_device() != dev \
                    or not v[0].is_contiguous():
                _bad_vector(*v, dev)
    os, qs = _rows(out, "out"), _rows(query, "query")
    if not (out.get_device() == dev and key_cache.get_device() == dev
            and value_cache.get_device() == dev and block_table.get_device() == dev
            and (workspace is None or workspace.get_device() == dev)):
        _bad_device("out, caches, block_table or workspace", dev)
    max_context_len = _bound(max_context_len, "max_context_len")
    max_prefix_len = _bound(max_prefix_len, "max_prefix_len")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if d_error is not None:
        _check_error(d_error, dev)
    _current(dev)
    if workspace is None:
        need = pa_decode_shared_plan(s, g, hq, hkv, d, max_context_len, max_prefix_len, lib=lib)
        # on the call's stream: a later allocation of another one must not get it
        with torch.cuda.stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    st = lib.pa_decode_shared(
        out.data_ptr(), os, query.data_ptr(), qs, key_cache.data_ptr(), value_cache.data_ptr(),
        block_table.data_ptr(), stride if s > 1 else width, width, context_lens.data_ptr(),
        group_starts.data_ptr(), prefix_lens.data_ptr(), g, s, hq, hkv, d, bs, nb, float(scale),
        max_context_len, max_prefix_len, workspace.data_ptr(),
        workspace.nbytes, _DTYPE[dtype], None if d_error is None else d_error.data_ptr(),
        _raw_stream(stream, dev))
    if st:
        _check(lib, st, "pa_decode_shared")
    return out
