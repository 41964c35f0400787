"""Thin torch binding of the C ABI (argument marshalling only).

Every function checks dtypes, devices and contiguity, passes raw pointers and
the current CUDA stream to libpa, and raises ``PagedAttentionError`` on a
non-zero status.  No arithmetic of the attention path happens here.
"""
from __future__ import annotations

import array
import collections
import ctypes
import functools
import math
import operator
import threading

import numpy as np
import torch

from . import _lib

PA_OK = 0


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def _check(status: int, lib=None):
    if status != PA_OK:
        lib = lib or _lib.load()
        msg = lib.pa_last_error().decode(errors="replace")
        name = lib.pa_status_string(status).decode()
        raise PagedAttentionError(status, f"{name}: {msg}")


# The raw handle of the current stream of a device index; without it (another
# torch) through the Stream object, 2 us instead of 0.1.  The current device
# without the public function's check that CUDA is initialised.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(t: torch.Tensor | None = None) -> int:
    if t is not None and t.is_cuda and _raw_stream is not None:
        return _raw_stream(t.get_device())
    dev = t.device if t is not None else None
    return torch.cuda.current_stream(dev).cuda_stream


def _call(fn, t: torch.Tensor, *args):
    """fn(*args, current stream) of libpa with t's device current."""
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    index = t.get_device()
    stream = _raw_stream(index) if _raw_stream is not None else _stream(t)
    if index == _current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != PA_OK:
        _check(status)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, device=None, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


PA_KV_BF16, PA_KV_FP8_E4M3, PA_KV_FP4 = 0, 1, 2
_FP8_DTYPES = (torch.uint8,) + ((torch.float8_e4m3fn,) if hasattr(torch, "float8_e4m3fn") else ())


def _need_at_least(t: torch.Tensor | None, name: str, n: int):
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} must hold at least {n} elements")


def _kv_dtype(k_cache: torch.Tensor, v_cache: torch.Tensor, asked: int | None = None) -> int:
    """PA_KV_BF16 for bf16 pools, PA_KV_FP8_E4M3 for E4M3 codes (uint8 or
    torch.float8_e4m3fn); PA_KV_FP4 only where the caller asks for it (4-bit
    rows are uint8 as well)."""
    if k_cache.dtype != v_cache.dtype:
        raise TypeError("k_cache and v_cache dtypes differ")
    if asked is not None and asked not in (PA_KV_BF16, PA_KV_FP8_E4M3, PA_KV_FP4):
        raise ValueError(f"kv_dtype {asked} is not PA_KV_BF16, PA_KV_FP8_E4M3 or PA_KV_FP4")
    if asked == PA_KV_FP4:
        if k_cache.dtype != torch.uint8:
            raise TypeError(f"4-bit pools are uint8 rows, got {k_cache.dtype}")
        return PA_KV_FP4
    found = _kv_dtype_of(k_cache)
    if asked is not None and asked != found:
        raise TypeError(f"kv_dtype {asked} does not match pools of {k_cache.dtype}")
    return found


def _kv_dtype_of(k_cache: torch.Tensor) -> int:
    if k_cache.dtype == torch.bfloat16:
        return PA_KV_BF16
    if k_cache.dtype in _FP8_DTYPES:
        return PA_KV_FP8_E4M3
    raise TypeError(f"pools must be bf16 or E4M3 (uint8 / float8_e4m3fn), got {k_cache.dtype}")


def _need_scales(k_scale, v_scale, Hkv: int, dev):
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is None:
            raise ValueError(f"{n} is required for FP8 and 4-bit pools")
        _need(t, n, torch.float32, dev)
        if t.numel() != Hkv:
            raise ValueError(f"{n} must hold one scale per KV head ({Hkv})")


def abi_version() -> int:
    return int(_lib.load().pa_abi_version())


# Device error bits (include/pa.h, PA_DEVERR_*).
PA_DEVERR_PAGE_RANGE = 1
PA_DEVERR_SEQLENS = 2
PA_DEVERR_TIMEOUT = 4
PA_DEVERR_POSITION = 8
PA_DEVERR_TABLE_INDEX = 16
PA_DEVERR_NO_PAGES = 32


def device_error() -> int:
    """Read and clear the device error word (synchronises the current stream).

    A launch whose bounded wait gave up (PA_DEVERR_TIMEOUT) may leave its
    scheduler counters non-zero, and the next launch sharing the array would
    skip work items: the scheduler arrays cached by ``prefill_scheduler``
    are cleared then (after the device has drained)."""
    lib = _lib.load()
    bits = ctypes.c_int32(0)
    _check(lib.pa_device_error(ctypes.byref(bits), _stream()), lib)
    if bits.value & PA_DEVERR_TIMEOUT:
        _reset_schedulers()
    return int(bits.value)


def store_kv(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
             k_cache: torch.Tensor, v_cache: torch.Tensor) -> None:
    """Write token t's K/V rows into row slot_mapping[t] of the pools.
    k, v: bf16 [T, Hkv, d]; caches: bf16 [num_pages, page_size, Hkv, d] or
    [num_slots, Hkv, d]; slot_mapping: int32 [T] (negative = skip)."""
    dev = k_cache.device
    for t, n in ((k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, dev)
    _need(slot_mapping, "slot_mapping", torch.int32, dev)
    Hkv, d = k_cache.shape[-2], k_cache.shape[-1]
    T = slot_mapping.numel()
    if k.numel() != T * Hkv * d or v.numel() != T * Hkv * d:
        raise ValueError("k/v must hold num_tokens rows of Hkv*d")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    num_slots = k_cache.numel() // (Hkv * d)
    lib = _lib.load()
    _check(lib.pa_store_kv(_ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(k_cache), _ptr(v_cache),
                           num_slots, Hkv, d, _stream(k_cache)), lib)


def store_kv_fp8(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor) -> None:
    """Write token t's K/V rows into row slot_mapping[t] of E4M3 pools:
    code = E4M3(x / scale[kv head]).  k, v: bf16 [T, Hkv, d]; caches: uint8
    or float8_e4m3fn [num_pages, page_size, Hkv, d] or [num_slots, Hkv, d];
    k_scale, v_scale: fp32 [Hkv]."""
    dev = k_cache.device
    for t, n in ((k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, dev)
    if _kv_dtype(k_cache, v_cache) != PA_KV_FP8_E4M3:
        raise TypeError("store_kv_fp8 needs E4M3 pools")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, k_cache.dtype, dev)
    _need(slot_mapping, "slot_mapping", torch.int32, dev)
    Hkv, d = k_cache.shape[-2], k_cache.shape[-1]
    _need_scales(k_scale, v_scale, Hkv, dev)
    T = slot_mapping.numel()
    if k.numel() != T * Hkv * d or v.numel() != T * Hkv * d:
        raise ValueError("k/v must hold num_tokens rows of Hkv*d")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    num_slots = k_cache.numel() // (Hkv * d)
    lib = _lib.load()
    _check(lib.pa_store_kv_fp8(_ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(k_cache), _ptr(v_cache),
                               num_slots, Hkv, d, _ptr(k_scale), _ptr(v_scale), _stream(k_cache)), lib)


@functools.lru_cache(maxsize=None)
def _fp4_row_bytes(num_kv_heads: int, head_dim: int) -> int:
    lib = _lib.load()
    n = int(lib.pa_fp4_row_bytes(num_kv_heads, head_dim))
    if n == 0:
        raise ValueError(lib.pa_last_error().decode(errors="replace"))
    return n


def fp4_row_bytes(num_kv_heads: int, head_dim: int) -> int:
    """Bytes of one token's row in a 4-bit pool of K (or of V): a pool is a
    uint8 tensor [num_pages, page_size, fp4_row_bytes(Hkv, d)]."""
    return _fp4_row_bytes(int(num_kv_heads), int(head_dim))


def _fp4_pools(k_cache, v_cache, k_scale, v_scale, Hkv: int, d: int, dev) -> int:
    """Checks a pair of 4-bit pools for Hkv heads of size d; returns their
    slots."""
    _need(k_cache, "k_cache", torch.uint8, dev)
    _need(v_cache, "v_cache", torch.uint8, dev)
    _need_scales(k_scale, v_scale, Hkv, dev)
    shape, row = k_cache.shape, _fp4_row_bytes(Hkv, d)
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache shapes differ")
    if len(shape) not in (2, 3) or shape[-1] != row:
        raise ValueError(f"a 4-bit pool of {Hkv} heads of size {d} is [num_pages, page_size, {row}] bytes, got "
                         f"{tuple(shape)}")
    return k_cache.numel() // row


def store_kv_fp4(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor) -> None:
    """Write token t's K/V rows into row slot_mapping[t] of 4-bit pools (E2M1
    codes with an E4M3 scale per 16 elements and an fp32 scale per head).  k,
    v: bf16 [T, Hkv, d], d 64 or 128; caches: uint8 [num_pages, page_size,
    fp4_row_bytes(Hkv, d)] or [num_slots, row bytes]; k_scale, v_scale: fp32
    [Hkv], best the head's largest magnitude / 2688.  A negative slot is
    skipped."""
    dev = k_cache.device
    _need(k, "k", torch.bfloat16, dev)
    _need(v, "v", torch.bfloat16, dev)
    _need(slot_mapping, "slot_mapping", torch.int32, dev)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or slot_mapping.numel() != shape[0]:
        raise ValueError("k and v must be [T, Hkv, d] with one slot per token")
    T, Hkv, d = shape
    slots = _fp4_pools(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev)
    _call(_lib.load().pa_store_kv_fp4, k_cache, k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), T,
          k_cache.data_ptr(), v_cache.data_ptr(), slots, Hkv, d, k_scale.data_ptr(), v_scale.data_ptr())


def load_kv_fp4(slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                v_scale: torch.Tensor, head_dim: int, *, k_out: torch.Tensor | None = None,
                v_out: torch.Tensor | None = None):
    """The rows ``slots`` (int32 [T]) of 4-bit pools as bf16 (k, v), each
    [T, Hkv, head_dim]; Hkv is the number of scales.  A negative slot gives
    zeros."""
    dev = k_cache.device
    _need(slots, "slots", torch.int32, dev)
    if k_scale is None:
        raise ValueError("k_scale is required for FP8 and 4-bit pools")
    T, Hkv, d = slots.numel(), k_scale.numel(), int(head_dim)
    num_slots = _fp4_pools(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev)
    shape = (T, Hkv, d)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _need(k_out, "k_out", torch.bfloat16, dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _need(v_out, "v_out", torch.bfloat16, dev)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"k_out and v_out must be [{T}, {Hkv}, {d}]")
    _call(_lib.load().pa_load_kv_fp4, k_cache, slots.data_ptr(), T, k_cache.data_ptr(), v_cache.data_ptr(), num_slots,
          Hkv, d, k_scale.data_ptr(), v_scale.data_ptr(), k_out.data_ptr(), v_out.data_ptr())
    return k_out, v_out


def rope_cos_sin_table(max_pos: int, rot_dim: int, base: float = 10000.0) -> torch.Tensor:
    """Host fp32 [max_pos, rot_dim] rotary table (cos of the rot_dim/2 angles
    p * base^(-2i/rot_dim), then their sin), computed by the C library."""
    t = torch.empty((int(max_pos), int(rot_dim)), dtype=torch.float32)
    lib = _lib.load()
    _check(lib.pa_rope_cos_sin_table(t.data_ptr() if t.numel() else None, int(max_pos), int(rot_dim),
                                     float(base)), lib)
    return t


def rope_store_kv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                  cos_sin: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, *, q_out: torch.Tensor | None = None,
                  interleaved: bool = False, k_scale: torch.Tensor | None = None,
                  v_scale: torch.Tensor | None = None, kv_dtype: int | None = None) -> torch.Tensor:
    """Rotary embedding of q and k at ``positions`` fused with the K/V store.
    q bf16 [T, Hq, d]; k, v bf16 [T, Hkv, d]; cos_sin fp32 [max_pos, rot_dim]
    on the device; pools bf16 or E4M3 (with ``k_scale``/``v_scale``), or with
    ``kv_dtype=PA_KV_FP4`` 4-bit rows (``store_kv_fp4``).  Returns the rotated
    q (``q_out``, which may be ``q``)."""
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, dev)
    _need(positions, "positions", torch.int32, dev)
    _need(slot_mapping, "slot_mapping", torch.int32, dev)
    _need(cos_sin, "cos_sin", torch.float32, dev)
    kvd = _kv_dtype(k_cache, v_cache, kv_dtype)
    T, Hq, d = q.shape
    if kvd == PA_KV_FP4:
        if k.dim() != 3:
            raise ValueError("k must be [T, Hkv, d]")
        Hkv = k.shape[1]
        _fp4_pools(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev)
    else:
        for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, n, k_cache.dtype, dev)
        Hkv = k_cache.shape[-2]
    if (kvd != PA_KV_FP4 and k_cache.shape[-1] != d) or k.numel() != T * Hkv * d or v.numel() != T * Hkv * d:
        raise ValueError("k/v/pool shapes do not match q")
    if positions.numel() != T or slot_mapping.numel() != T:
        raise ValueError("positions and slot_mapping must hold one entry per token")
    if kvd == PA_KV_FP8_E4M3:
        _need_scales(k_scale, v_scale, Hkv, dev)
    if q_out is None:
        q_out = torch.empty_like(q)
    _need(q_out, "q_out", torch.bfloat16, dev)
    _need_at_least(q_out, "q_out", q.numel())
    p = _lib.RopeStoreParams(
        q=_ptr(q), q_out=_ptr(q_out), k=_ptr(k), v=_ptr(v), positions=_ptr(positions),
        cos_sin=_ptr(cos_sin), max_pos=cos_sin.shape[0], rot_dim=cos_sin.shape[1],
        interleaved=int(bool(interleaved)), slot_mapping=_ptr(slot_mapping), num_tokens=T,
        num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, k_cache=_ptr(k_cache), v_cache=_ptr(v_cache),
        num_slots=k_cache.numel() // (k_cache.shape[-1] if kvd == PA_KV_FP4 else Hkv * d), kv_dtype=kvd,
        k_scale=_ptr(k_scale) if kvd != PA_KV_BF16 else None,
        v_scale=_ptr(v_scale) if kvd != PA_KV_BF16 else None)
    _call(_lib.load().pa_rope_store_kv, q, ctypes.byref(p))
    return q_out


def build_seqlens(cached_len, extend_len):
    """Host metadata: (cu_seqlens_q, cu_seqlens_k, cache_seqlens, max_q, max_k)
    as int32 numpy arrays (the C entry point does the arithmetic)."""
    c = np.ascontiguousarray(cached_len, dtype=np.int32)
    e = np.ascontiguousarray(extend_len, dtype=np.int32)
    B = c.shape[0]
    cu_q = np.zeros(B + 1, np.int32)
    cu_k = np.zeros(B + 1, np.int32)
    cs = np.zeros(max(B, 1), np.int32)
    mq = ctypes.c_int32(0)
    mk = ctypes.c_int32(0)
    lib = _lib.load()
    _check(lib.pa_build_seqlens(c.ctypes.data, e.ctypes.data, B, cu_q.ctypes.data,
                                cu_k.ctypes.data, cs.ctypes.data, ctypes.byref(mq),
                                ctypes.byref(mk)), lib)
    return cu_q, cu_k, cs[:B], int(mq.value), int(mk.value)


def build_page_table(token_table: torch.Tensor, table_idx: torch.Tensor, max_seqlen_k: int,
                     page_size: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Device metadata: page table [B, ceil(max_seqlen_k / page_size)] from the
    token-granular global table (sliced with step page_size, floor-divided)."""
    dev = token_table.device
    _need(token_table, "token_table", torch.int32, dev)
    _need(table_idx, "table_idx", torch.int32, dev)
    B = table_idx.numel()
    ncols = -(-int(max_seqlen_k) // int(page_size))
    if token_table.dim() != 2 or token_table.stride(1) != 1:
        raise ValueError("token_table must be 2-D with unit column stride")
    if out is None:
        out = torch.empty((B, max(ncols, 1)), dtype=torch.int32, device=dev)
    _need(out, "out", torch.int32, dev, contiguous=False)
    if out.dim() != 2 or out.stride(1) != 1 or out.shape[0] < B or out.shape[1] < ncols:
        raise ValueError(f"out must be 2-D with unit column stride and at least [{B}, {ncols}]")
    lib = _lib.load()
    _check(lib.pa_build_page_table(_ptr(token_table), token_table.stride(0), token_table.shape[0],
                                   _ptr(table_idx), B,
                                   int(max_seqlen_k), int(page_size), _ptr(out), out.stride(0),
                                   _stream(token_table)), lib)
    return out


def build_batch(cached_len: torch.Tensor, extend_len: torch.Tensor, token_table: torch.Tensor, table_idx: torch.Tensor,
                page_size: int, max_seqlen_k: int, *, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                cache_seqlens: torch.Tensor, positions: torch.Tensor, slot_mapping: torch.Tensor,
                page_table: torch.Tensor, totals: torch.Tensor, free_pages: torch.Tensor | None = None,
                free_cursor: torch.Tensor | None = None) -> None:
    """A batch's metadata from lengths on the device, in one launch
    (``pa_build_batch``; ``metadata.BatchPlanner`` owns the outputs).
    cached_len, extend_len, table_idx: int32 [B]; token_table: int32 [rows, >=
    max_seqlen_k].  Outputs: cu_seqlens_q, cu_seqlens_k [B+1], cache_seqlens
    [B], positions and slot_mapping [T] (padded with 0 and -1 past the batch's
    tokens), page_table [>= B, >= ceil(max_seqlen_k / page_size)] (columns past
    a request's pages are left as they were), totals [4] (new tokens, longest
    extend, longest length, new pages).  ``free_pages`` (int32): take the new
    tokens' pages from its first entries and enter their slots in
    ``token_table``; the caller moves the list on by totals[3] before the next
    call.  With ``free_cursor`` (int32 [2] on the device, zeros at first) they
    are taken from entry free_cursor[0] on, which the call moves on itself
    (``pa_build_batch_from``): a captured call needs it."""
    dev = token_table.device
    B = cached_len.numel()
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k"), (cache_seqlens, "cache_seqlens"),
                 (positions, "positions"), (slot_mapping, "slot_mapping"), (totals, "totals")):
        _need(t, n, torch.int32, dev)
    _need_rows(page_table, "page_table", dev)
    max_k, P = int(max_seqlen_k), int(page_size)
    if P <= 0:
        raise ValueError("page_size must be positive")
    if cu_seqlens_q.numel() < B + 1 or cu_seqlens_k.numel() < B + 1 or cache_seqlens.numel() < B or totals.numel() < 4:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must hold B + 1 entries, cache_seqlens B, totals 4")
    if positions.numel() != slot_mapping.numel():
        raise ValueError("positions and slot_mapping must have the same size")
    if page_table.shape[0] < B or page_table.shape[1] < -(-max_k // P):
        raise ValueError(f"page_table must be at least [{B}, {-(-max_k // P)}]")
    out = _BatchOut(cu_seqlens_q, cu_seqlens_k, cache_seqlens, positions, slot_mapping, page_table, totals)
    _build_batch(cached_len, extend_len, token_table, table_idx, P, max_k, out, free_pages, free_cursor)


_BatchOut = collections.namedtuple("_BatchOut", "cu_seqlens_q cu_seqlens_k cache_seqlens positions slot_mapping "
                                                "page_table totals")


def _need_rows(t, name, dev):
    _need(t, name, torch.int32, dev, contiguous=False)
    if t.dim() != 2 or t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name} must be 2-D with unit column stride and rows that do not overlap")


def _build_batch(cached_len, extend_len, token_table, table_idx, page_size, max_seqlen_k, out, free_pages, free_cursor):
    """build_batch into checked outputs (the attributes of ``out``)."""
    dev = out.totals.device
    _need(cached_len, "cached_len", torch.int32, dev)
    _need(extend_len, "extend_len", torch.int32, dev)
    _need(table_idx, "table_idx", torch.int32, dev)
    _need_rows(token_table, "token_table", dev)
    if free_pages is not None:
        _need(free_pages, "free_pages", torch.int32, dev)
    if free_cursor is not None:
        _need(free_cursor, "free_cursor", torch.int32, dev)
        if free_pages is None:
            raise ValueError("free_cursor needs free_pages")
        if free_cursor.numel() < 2:
            raise ValueError("free_cursor must hold 2 int32")
    B, width = cached_len.numel(), token_table.shape[1]
    if extend_len.numel() != B or table_idx.numel() != B:
        raise ValueError("cached_len, extend_len and table_idx must hold one entry per request")
    if width < max_seqlen_k:
        raise ValueError(f"token_table must be at least {max_seqlen_k} wide")
    pt = out.page_table
    # an empty list is a list all the same: NULL would mean none
    free_ptr = None if free_pages is None else free_pages.data_ptr() or out.totals.data_ptr()
    p = _lib.BatchParams(
        cached_len.data_ptr(), extend_len.data_ptr(), B, max_seqlen_k, page_size, token_table.data_ptr(),
        max(token_table.stride(0), width), token_table.shape[0], table_idx.data_ptr(), free_ptr,
        0 if free_pages is None else free_pages.numel(), out.positions.numel(), out.cu_seqlens_q.data_ptr(),
        out.cu_seqlens_k.data_ptr(), out.cache_seqlens.data_ptr(), out.positions.data_ptr(), out.slot_mapping.data_ptr(),
        pt.data_ptr(), max(pt.stride(0), pt.shape[1]), out.totals.data_ptr())
    _call(_lib.load().pa_build_batch_from, out.totals, ctypes.byref(p), _ptr(free_cursor))


def _pool_geometry(k_cache: torch.Tensor, v_cache: torch.Tensor, page_size: int | None):
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    if k_cache.dim() == 4:
        num_pages, P, Hkv, d = k_cache.shape
        if page_size is not None and page_size != P:
            raise ValueError("page_size does not match the pool shape")
    elif k_cache.dim() == 3:
        if page_size is None:
            raise ValueError("page_size is required for a [slots, Hkv, d] pool")
        slots, Hkv, d = k_cache.shape
        P = page_size
        num_pages = slots // P
    else:
        raise ValueError("pool must be [pages, page_size, Hkv, d] or [slots, Hkv, d]")
    return int(num_pages), int(P), int(Hkv), int(d)


def _fp4_geometry(k_cache, v_cache, page_size, k_scale, v_scale, d: int, dev):
    """_pool_geometry of 4-bit pools [pages, page_size, row bytes] or [slots,
    row bytes]; the heads are counted by the scales."""
    if k_scale is None:
        raise ValueError("k_scale is required for FP8 and 4-bit pools")
    Hkv = k_scale.numel()
    slots = _fp4_pools(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev)
    shape = k_cache.shape
    if len(shape) == 3:
        if page_size is not None and page_size != shape[1]:
            raise ValueError("page_size does not match the pool shape")
        return shape[0], shape[1], Hkv, d
    if page_size is None:
        raise ValueError("page_size is required for a [slots, row bytes] pool")
    return slots // int(page_size), int(page_size), Hkv, d


# Zeroed scheduler arrays of pa_prefill, one per (device, stream): launches on
# one stream run one after the other, so they can share one array (each
# launch leaves it at zero); launches on different streams get their own.
_sched_lock = threading.Lock()
_sched_arrays: dict = {}
PA_PREFILL_SCHEDULER_INTS = 2
PA_MIXED_SCHEDULER_INTS = 4


def _reset_schedulers() -> None:
    """Zero every cached scheduler array once the work in flight has ended."""
    with _sched_lock:
        arrays = list(_sched_arrays.values())
    for t in arrays:
        if t.is_cuda:
            torch.cuda.synchronize(t.device)
        t.zero_()
        if t.is_cuda:
            torch.cuda.synchronize(t.device)


def prefill_scheduler(device=None, stream=None) -> torch.Tensor:
    """The cached zeroed int32 [4] scheduler array for (device, stream):
    the default of ``prefill(scheduler=None)`` and ``mixed_batch``.  Create
    it before capturing a CUDA graph that calls either on that stream."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    key = (dev.index, int(stream.cuda_stream))
    with _sched_lock:
        t = _sched_arrays.get(key)
        if t is None:
            t = torch.zeros(PA_MIXED_SCHEDULER_INTS, dtype=torch.int32, device=dev)
            _sched_arrays[key] = t
        return t


def prefill(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
            cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_seqlen_q: int,
            max_seqlen_k: int, *, causal: bool = True, scale: float | None = None,
            page_size: int | None = None, out: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, k_scale: torch.Tensor | None = None,
            v_scale: torch.Tensor | None = None, sliding_window: int = 0,
            max_ctas: int = 0, scheduler: torch.Tensor | None = None,
            block_mask: torch.Tensor | None = None, kv_dtype: int | None = None) -> torch.Tensor:
    """Varlen prefill / extend attention.  q: bf16 [total_q, Hq, d];
    returns out bf16 [total_q, Hq, d]; lse (optional) fp32 [Hq, total_q].
    Pools are bf16, or E4M3 codes (uint8 / float8_e4m3fn) with fp32
    per-KV-head ``k_scale`` and ``v_scale``, or, with ``kv_dtype=PA_KV_FP4``,
    4-bit rows with such scales (``store_kv_fp4``); on those q is rounded to
    f16, so |q| must stay below 65504.  ``scheduler`` is the int32 [2]
    work-counter array of the launch (zero between launches); by default the
    array cached for the current stream (``prefill_scheduler``).
    ``block_mask``: optional uint8 [B, nq, nk] on the device; entry
    [b, i // 128, j // 128] == 0 hides key j from request b's query row i
    (rows counted from the request's first row)."""
    p, out = _prefill_params(q, k_cache, v_cache, page_table, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                             max_seqlen_k, causal, scale, page_size, out, lse, k_scale, v_scale, sliding_window,
                             max_ctas, scheduler, block_mask, PA_PREFILL_SCHEDULER_INTS, kv_dtype)
    _call(_lib.load().pa_prefill, q, ctypes.byref(p))
    return out


def _prefill_params(q, k_cache, v_cache, page_table, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                    causal, scale, page_size, out, lse, k_scale, v_scale, sliding_window, max_ctas, scheduler,
                    block_mask, sched_ints, kv_dtype=None):
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    kvd = _kv_dtype(k_cache, v_cache, kv_dtype)
    if kvd == PA_KV_FP4:
        num_pages, P, Hkv, d = _fp4_geometry(k_cache, v_cache, page_size, k_scale, v_scale, q.shape[-1],
                                                  q.device)
    else:
        num_pages, P, Hkv, d = _pool_geometry(k_cache, v_cache, page_size)
    if kvd != PA_KV_FP4:                              # (4-bit pools: _fp4_geometry)
        for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, n, k_cache.dtype, dev)
    if kvd == PA_KV_FP8_E4M3:
        _need_scales(k_scale, v_scale, Hkv, dev)
    for t, n in ((page_table, "page_table"), (cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k")):
        _need(t, n, torch.int32, dev, contiguous=(n != "page_table"))
    if page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be 2-D with unit column stride")
    total_q, Hq, dq = q.shape
    if dq != d:
        raise ValueError("head_dim of q and the pool differ")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, dev)
    if kvd == PA_KV_FP4:
        _need_at_least(out, "out", q.numel())
        if not page_table.shape[0] + 1 >= cu_seqlens_k.numel() == cu_seqlens_q.numel() >= 1:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must hold num_seqs + 1 entries, page_table a row per sequence")
    if lse is not None:
        _need(lse, "lse", torch.float32, dev, contiguous=False)
        if lse.dim() != 2 or lse.shape[0] != Hq or lse.stride(1) != 1:
            raise ValueError("lse must be [Hq, >= total_q] with unit inner stride")
        if kvd == PA_KV_FP4 and lse.shape[1] < total_q:
            raise ValueError("lse must be [Hq, >= total_q] with unit inner stride")
    if block_mask is not None:
        _need(block_mask, "block_mask", torch.uint8, dev)
        if block_mask.dim() != 3 or block_mask.shape[0] != cu_seqlens_q.numel() - 1:
            raise ValueError("block_mask must be [num_seqs, q_blocks, k_blocks]")
    if scheduler is None:
        scheduler = _sched_arrays.get((dev.index, _stream(q)))
        if scheduler is None:
            scheduler = prefill_scheduler(dev)
    else:
        _need(scheduler, "scheduler", torch.int32, dev)
        if scheduler.numel() < sched_ints:
            raise ValueError(f"scheduler must hold {sched_ints} int32")
    p = _lib.PrefillParams(
        q=_ptr(q), k_cache=_ptr(k_cache), v_cache=_ptr(v_cache), page_table=_ptr(page_table),
        page_table_stride=page_table.stride(0), total_q=total_q, cu_seqlens_q=_ptr(cu_seqlens_q),
        cu_seqlens_k=_ptr(cu_seqlens_k), num_seqs=cu_seqlens_q.numel() - 1,
        max_seqlen_q=int(max_seqlen_q), max_seqlen_k=int(max_seqlen_k), num_q_heads=Hq,
        num_kv_heads=Hkv, head_dim=d, page_size=P, num_pages=num_pages, causal=int(bool(causal)),
        scale=float(1.0 / math.sqrt(d) if scale is None else scale), out=_ptr(out),
        lse=_ptr(lse), lse_stride=(lse.stride(0) if lse is not None else 0), kv_dtype=kvd,
        k_scale=_ptr(k_scale) if kvd != PA_KV_BF16 else None,
        v_scale=_ptr(v_scale) if kvd != PA_KV_BF16 else None, sliding_window=int(sliding_window),
        max_ctas=int(max_ctas), scheduler=_ptr(scheduler), block_mask=_ptr(block_mask),
        block_mask_q_blocks=int(block_mask.shape[1]) if block_mask is not None else 0,
        block_mask_k_blocks=int(block_mask.shape[2]) if block_mask is not None else 0)
    return p, out


def _decode_params(q, k_cache, v_cache, page_table, cache_seqlens, max_seqlen_k, scale, page_size,
                   out, lse, workspace, kv_chunk, k_scale=None, v_scale=None, sliding_window=0,
                   max_ctas=0, overlap_previous=False, kv_dtype=None):
    kvd = _kv_dtype(k_cache, v_cache, kv_dtype)
    if kvd == PA_KV_FP4:
        num_pages, P, Hkv, d = _fp4_geometry(k_cache, v_cache, page_size, k_scale, v_scale, q.shape[-1],
                                                  q.device)
    else:
        num_pages, P, Hkv, d = _pool_geometry(k_cache, v_cache, page_size)
    B, Hq, dq = q.shape
    if dq != d:
        raise ValueError("head_dim of q and the pool differ")
    if kvd == PA_KV_FP8_E4M3:
        _need_scales(k_scale, v_scale, Hkv, q.device)
    if kvd == PA_KV_FP4:
        _need_at_least(cache_seqlens, "cache_seqlens", B)
        _need_at_least(out, "out", q.numel())
        _need_at_least(lse, "lse", B * Hq)
        if page_table.shape[0] < B:
            raise ValueError("page_table must have a row per sequence")
    return _lib.DecodeParams(
        q=_ptr(q), k_cache=_ptr(k_cache), v_cache=_ptr(v_cache), page_table=_ptr(page_table),
        page_table_stride=page_table.stride(0) if page_table is not None else 0,
        cache_seqlens=_ptr(cache_seqlens), num_seqs=B, max_seqlen_k=int(max_seqlen_k),
        num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, page_size=P, num_pages=num_pages,
        scale=float(1.0 / math.sqrt(d) if scale is None else scale), out=_ptr(out), lse=_ptr(lse),
        workspace=_ptr(workspace), workspace_bytes=(workspace.numel() * workspace.element_size()
                                                    if workspace is not None else 0),
        kv_chunk=int(kv_chunk), kv_dtype=kvd,
        k_scale=_ptr(k_scale) if kvd != PA_KV_BF16 else None,
        v_scale=_ptr(v_scale) if kvd != PA_KV_BF16 else None, sliding_window=int(sliding_window),
        max_ctas=int(max_ctas), overlap_previous=int(bool(overlap_previous)))


def _decode_sizes(q_shape, k_cache, max_seqlen_k, page_size, kv_chunk, kv_dtype, num_kv_heads):
    """The host fields that the decode's split layout depends on."""
    B, Hq, d = q_shape
    if kv_dtype == PA_KV_FP4:
        if num_kv_heads is None:
            raise ValueError("num_kv_heads is required for 4-bit pools")
        if k_cache.dim() == 2 and page_size is None:
            raise ValueError("page_size is required for a [slots, row bytes] pool")
        P = int(k_cache.shape[1] if k_cache.dim() == 3 else page_size)
        num_pages, Hkv = k_cache.numel() // (k_cache.shape[-1] * P), int(num_kv_heads)
    else:
        kv_dtype = PA_KV_BF16                         # FP8 pools split alike
        num_pages, P, Hkv, _ = _pool_geometry(k_cache, k_cache, page_size)
    return _lib.DecodeParams(num_seqs=B, max_seqlen_k=int(max_seqlen_k), num_q_heads=Hq,
                             num_kv_heads=Hkv, head_dim=d, page_size=P, num_pages=num_pages,
                             scale=1.0, kv_chunk=int(kv_chunk), kv_dtype=kv_dtype)


def decode_workspace_size(q_shape, k_cache: torch.Tensor, max_seqlen_k: int, *,
                          page_size: int | None = None, kv_chunk: int = 0, kv_dtype: int | None = None,
                          num_kv_heads: int | None = None) -> int:
    """Workspace bytes pa_decode needs (0 when a single split suffices).
    4-bit pools need ``kv_dtype=PA_KV_FP4`` and ``num_kv_heads``."""
    p = _decode_sizes(q_shape, k_cache, max_seqlen_k, page_size, kv_chunk, kv_dtype, num_kv_heads)
    return int(_lib.load().pa_decode_workspace_size(ctypes.byref(p)))


def decode_kv_chunk(q_shape, k_cache: torch.Tensor, max_seqlen_k: int, *,
                    page_size: int | None = None, kv_chunk: int = 0, kv_dtype: int | None = None,
                    num_kv_heads: int | None = None) -> int:
    p = _decode_sizes(q_shape, k_cache, max_seqlen_k, page_size, kv_chunk, kv_dtype, num_kv_heads)
    return int(_lib.load().pa_decode_kv_chunk(ctypes.byref(p)))


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
           cache_seqlens: torch.Tensor, max_seqlen_k: int, *, scale: float | None = None,
           page_size: int | None = None, out: torch.Tensor | None = None,
           lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
           kv_chunk: int = 0, k_scale: torch.Tensor | None = None,
           v_scale: torch.Tensor | None = None, sliding_window: int = 0,
           max_ctas: int = 0, overlap_previous: bool = False, kv_dtype: int | None = None) -> torch.Tensor:
    """Split-KV decode: q bf16 [B, Hq, d] -> out bf16 [B, Hq, d]; lse fp32 [B, Hq].
    Pools are bf16, or E4M3 codes (uint8 / float8_e4m3fn) with fp32 per-KV-head
    ``k_scale`` and ``v_scale``, or, with ``kv_dtype=PA_KV_FP4``, 4-bit rows
    with such scales (``store_kv_fp4``); on those q is rounded to f16, so |q|
    must stay below 65504.  ``workspace`` (a uint8 CUDA tensor) is allocated
    here when not given."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    kvd = _kv_dtype(k_cache, v_cache, kv_dtype)
    if kvd != PA_KV_FP4:                              # (4-bit pools: _fp4_geometry)
        for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, n, k_cache.dtype, dev)
    _need(cache_seqlens, "cache_seqlens", torch.int32, dev)
    _need(page_table, "page_table", torch.int32, dev, contiguous=False)
    if page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be 2-D with unit column stride")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", torch.bfloat16, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if workspace is None:
        need = decode_workspace_size(q.shape, k_cache, max_seqlen_k, page_size=page_size, kv_chunk=kv_chunk, kv_dtype=kvd,
                                     num_kv_heads=k_scale.numel() if kvd == PA_KV_FP4 and k_scale is not None else None)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    p = _decode_params(q, k_cache, v_cache, page_table, cache_seqlens, max_seqlen_k, scale, page_size,
                       out, lse, workspace, kv_chunk, k_scale, v_scale, sliding_window, max_ctas,
                       overlap_previous, kvd)
    _call(_lib.load().pa_decode, q, ctypes.byref(p))
    return out


def mixed_batch(q_prefill: torch.Tensor, q_decode: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                page_table_prefill: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                max_seqlen_q: int, max_seqlen_k_prefill: int, page_table_decode: torch.Tensor,
                cache_seqlens: torch.Tensor, max_seqlen_k_decode: int, *, causal: bool = True,
                scale: float | None = None, out_prefill: torch.Tensor | None = None,
                out_decode: torch.Tensor | None = None, lse_prefill: torch.Tensor | None = None,
                lse_decode: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                kv_chunk: int = 0, scheduler: torch.Tensor | None = None, prefill_ctas: int = 0,
                decode_sliding_window: int = 0, k_scale: torch.Tensor | None = None,
                v_scale: torch.Tensor | None = None):
    """One continuous batch in one launch (``pa_mixed_batch``): prefill /
    extend of ``q_prefill`` [total_q, Hq, d] (cu_seqlens_q/k, its page table)
    and decode of ``q_decode`` [B, Hq, d] (cache_seqlens, its page table)
    over the same bf16 pools.  ``prefill_ctas`` > 0: that many CTAs take
    prefill tiles before decode key ranges (the others start on decode at
    once); 0: the kernel chooses the count from the work of both halves.
    ``decode_sliding_window`` W > 0: each decode query sees its sequence's
    last W keys only (the prefill half takes no window).  FP8 (uint8 E4M3)
    pools take their per-KV-head ``k_scale`` / ``v_scale`` for both halves.
    Returns (out_prefill, out_decode)."""
    dev = q_prefill.device
    p, out_prefill = _prefill_params(q_prefill, k_cache, v_cache, page_table_prefill, cu_seqlens_q, cu_seqlens_k,
                                     max_seqlen_q, max_seqlen_k_prefill, causal, scale, None, out_prefill,
                                     lse_prefill, k_scale, v_scale, 0, int(prefill_ctas), scheduler, None,
                                     PA_MIXED_SCHEDULER_INTS)
    _need(q_decode, "q_decode", torch.bfloat16, dev)
    _need(cache_seqlens, "cache_seqlens", torch.int32, dev)
    _need(page_table_decode, "page_table_decode", torch.int32, dev, contiguous=False)
    if out_decode is None:
        out_decode = torch.empty_like(q_decode)
    need = decode_workspace_size(q_decode.shape, k_cache, max_seqlen_k_decode, kv_chunk=kv_chunk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    dp = _decode_params(q_decode, k_cache, v_cache, page_table_decode, cache_seqlens, max_seqlen_k_decode, scale,
                        None, out_decode, lse_decode, workspace, kv_chunk, k_scale, v_scale,
                        sliding_window=int(decode_sliding_window))
    lib = _lib.load()
    _check(lib.pa_mixed_batch(ctypes.byref(p), ctypes.byref(dp), _stream(q_prefill)), lib)
    return out_prefill, out_decode


def decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   page_table: torch.Tensor, cache_seqlens: torch.Tensor, max_seqlen_k: int, *,
                   scale: float | None = None, page_size: int | None = None,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   kv_chunk: int = 0, k_scale: torch.Tensor | None = None,
                   v_scale: torch.Tensor | None = None, sliding_window: int = 0,
                   kv_dtype: int | None = None) -> torch.Tensor:
    """Split-KV decode through ``pa_decode_noalloc``: the split partials go to
    the library's fixed 32 MiB device scratch, so no workspace is allocated
    (for callers that may not allocate device memory).  Calls on one device
    must not overlap on the GPU; sizes whose scratch would exceed 32 MiB raise
    PagedAttentionError.  ``out`` (and ``lse``) must be given by a caller that
    cannot allocate; they are created here only for convenience."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    kvd = _kv_dtype(k_cache, v_cache, kv_dtype)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, k_cache.dtype, dev)
    _need(cache_seqlens, "cache_seqlens", torch.int32, dev)
    _need(page_table, "page_table", torch.int32, dev, contiguous=False)
    if page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be 2-D with unit column stride")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    p = _decode_params(q, k_cache, v_cache, page_table, cache_seqlens, max_seqlen_k, scale, page_size,
                       out, lse, None, kv_chunk, k_scale, v_scale, sliding_window, kv_dtype=kvd)
    _call(_lib.load().pa_decode_noalloc, q, ctypes.byref(p))
    return out


def lse_combine(o_partial: torch.Tensor, lse_partial: torch.Tensor,
                splits_per_row: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None) -> torch.Tensor:
    """Merge split partials: o_partial fp32 [R, S, d], lse_partial fp32 [R, S]
    -> out bf16 [R, d] (and lse fp32 [R] if given)."""
    dev = o_partial.device
    _need(o_partial, "o_partial", torch.float32, dev)
    _need(lse_partial, "lse_partial", torch.float32, dev)
    R, S, d = o_partial.shape
    if lse_partial.shape != (R, S):
        raise ValueError("lse_partial must be [R, S]")
    if splits_per_row is not None:
        _need(splits_per_row, "splits_per_row", torch.int32, dev)
    if out is None:
        out = torch.empty((R, d), dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    lib = _lib.load()
    _check(lib.pa_lse_combine(_ptr(o_partial), _ptr(lse_partial), _ptr(splits_per_row), R, S, d,
                              _ptr(out), _ptr(lse), _stream(o_partial)), lib)
    return out


def _shared_bounds(B: int, max_seqlen_k: int, max_prefix, max_suffix, max_group):
    """The bounds of a decode over shared prefixes, by default the batch's own."""
    return (B if max_group is None else int(max_group), max_seqlen_k if max_prefix is None else int(max_prefix),
            max_seqlen_k if max_suffix is None else int(max_suffix))


def decode_shared_workspace_size(q_shape, k_cache: torch.Tensor, max_seqlen_k: int, num_groups: int, *,
                                 max_prefix: int | None = None, max_suffix: int | None = None, max_group: int | None = None,
                                 page_size: int | None = None, kv_chunk: int = 0, kv_dtype: int | None = None,
                                 num_kv_heads: int | None = None) -> int:
    """Workspace bytes of ``decode_shared`` for a batch of shape ``q_shape``
    in up to ``num_groups`` groups, under these bounds (``decode_shared`` says
    what they bound).  4-bit pools need ``kv_dtype=PA_KV_FP4`` and
    ``num_kv_heads``."""
    dec = _decode_sizes(q_shape, k_cache, max_seqlen_k, page_size, kv_chunk, kv_dtype, num_kv_heads)
    if kv_dtype != PA_KV_FP4:
        dec.kv_dtype = _kv_dtype(k_cache, k_cache, kv_dtype)
    bounds = _shared_bounds(int(q_shape[0]), int(max_seqlen_k), max_prefix, max_suffix, max_group)
    lib = _lib.load()
    need = int(lib.pa_decode_shared_workspace_size(ctypes.byref(_lib.DecodeSharedParams(dec, None, None, int(num_groups), *bounds))))
    if need == 0:
        raise ValueError(lib.pa_last_error().decode(errors="replace"))
    return need


def decode_shared(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                  cache_seqlens: torch.Tensor, max_seqlen_k: int, cu_groups: torch.Tensor, prefix_lens: torch.Tensor, *,
                  max_prefix: int | None = None, max_suffix: int | None = None, max_group: int | None = None,
                  scale: float | None = None, page_size: int | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, kv_chunk: int = 0,
                  k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                  kv_dtype: int | None = None) -> torch.Tensor:
    """``decode`` of a batch in which groups of consecutive sequences share
    their first keys; each group's prefix is read once (``pa_decode_shared``).
    q bf16 [B, Hq, d] -> out bf16 [B, Hq, d]; lse fp32 [B, Hq]; pools as for
    ``decode`` (over FP8 and 4-bit ones |q| must stay below 65504).  cu_groups: int32 [num_groups + 1], group g is sequences
    cu_groups[g] .. cu_groups[g+1] - 1; prefix_lens: int32 [B], the keys that
    sequence b shares with its group, equal within one, read through the
    page-table row of its first sequence, 0 for sequences behind the last
    group.  ``max_prefix`` and ``max_suffix`` bound the keys of a sequence in
    its prefix and behind it (default max_seqlen_k), ``max_group`` the
    sequences of a group (default B); tight bounds leave few CTAs idle."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    B, Hq, d = q.shape
    kvd = _kv_dtype(k_cache, v_cache, kv_dtype)
    if kvd == PA_KV_FP4:
        num_pages, P, Hkv, d = _fp4_geometry(k_cache, v_cache, page_size, k_scale, v_scale, d, dev)
    else:
        _need(k_cache, "k_cache", k_cache.dtype, dev)
        _need(v_cache, "v_cache", k_cache.dtype, dev)
        num_pages, P, Hkv, pool_d = _pool_geometry(k_cache, v_cache, page_size)
        if pool_d != d:
            raise ValueError("head_dim of q and the pool differ")
        if kvd == PA_KV_FP8_E4M3:
            _need_scales(k_scale, v_scale, Hkv, dev)
    _need(cache_seqlens, "cache_seqlens", torch.int32, dev)
    _need(cu_groups, "cu_groups", torch.int32, dev)
    _need(prefix_lens, "prefix_lens", torch.int32, dev)
    _need(page_table, "page_table", torch.int32, dev, False)
    max_k, groups = int(max_seqlen_k), cu_groups.numel() - 1
    if page_table.dim() != 2:
        raise ValueError("page_table must be 2-D with unit column stride")
    (rows, cols), (pt_stride, unit) = page_table.shape, page_table.stride()
    if unit != 1 or (rows > 1 and pt_stride < cols):
        raise ValueError("page_table must be 2-D with unit column stride and rows that do not overlap")
    if cache_seqlens.numel() != B or prefix_lens.numel() != B or rows < B:
        raise ValueError("cache_seqlens and prefix_lens must hold one entry per sequence, page_table a row")
    if cols * P < max_k:
        raise ValueError(f"page_table must have ceil({max_k} / {P}) columns")
    if groups < 0:
        raise ValueError("cu_groups must hold num_groups + 1 entries")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", torch.bfloat16, dev)
        if out.numel() != B * Hq * d:
            raise ValueError("out must have q's size")
    lse_ptr = None
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
        if lse.numel() != B * Hq:
            raise ValueError("lse must be [B, Hq]")
        lse_ptr = lse.data_ptr()
    bounds = _shared_bounds(B, max_k, max_prefix, max_suffix, max_group)
    if workspace is None:
        need = decode_shared_workspace_size(
            q.shape, k_cache, max_k, groups, max_group=bounds[0], max_prefix=bounds[1], max_suffix=bounds[2], page_size=page_size,
            kv_chunk=kv_chunk, kv_dtype=kvd, num_kv_heads=Hkv)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != q.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    ks = vs = None
    if kvd != PA_KV_BF16:
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    p = _lib.DecodeSharedParams(
        (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), max(pt_stride, cols), cache_seqlens.data_ptr(),
         B, max_k, Hq, Hkv, d, P, num_pages, 1.0 / math.sqrt(d) if scale is None else float(scale), out.data_ptr(), lse_ptr,
         workspace.data_ptr(), workspace.numel() * workspace.element_size(), int(kv_chunk), kvd, ks, vs),
        cu_groups.data_ptr(), prefix_lens.data_ptr(), groups, *bounds)
    _call(_lib.load().pa_decode_shared, q, ctypes.byref(p))
    return out


_LOGITS_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


@functools.lru_cache(maxsize=256)
def _select_workspace(groups: int, beams: int, vocab: int, num_out: int) -> int:
    lib = _lib.load()
    p = _lib.BeamSelectParams(num_groups=groups, beams=beams, vocab=vocab, num_out=num_out)
    need = int(lib.pa_beam_select_workspace_size(ctypes.byref(p)))
    message = lib.pa_last_error().decode(errors="replace")
    if message:
        raise ValueError(message)
    return need


def beam_select_workspace_size(num_groups: int, beams: int, vocab: int, num_out: int) -> int:
    """Workspace bytes of ``beam_select`` for these sizes and smaller ones."""
    return _select_workspace(int(num_groups), int(beams), int(vocab), int(num_out))


def beam_select(logits: torch.Tensor, scores: torch.Tensor, num_out: int | None = None, *,
                finished: torch.Tensor | None = None, pad_token: int = 0, out_scores: torch.Tensor | None = None,
                parents: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, out_finished: torch.Tensor | None = None):
    """Beam search's selection (``pa_beam_select``): per group the ``num_out``
    (default: the number of beams) largest of scores + log_softmax(logits)
    over beams and vocabulary.  logits: bf16, fp16 or fp32 [groups * beams, V]
    or [groups, beams, V], rows of unit stride at any distance; scores: fp32
    [groups, beams]; finished: uint8 or bool [groups, beams], non-zero for a
    beam that has ended (it offers itself, with ``pad_token``).  Returns
    (scores fp32, parents int32, tokens int32), each [groups, num_out], best
    first, equal totals by the lower beam, then the lower token; out_scores
    may be ``scores``.  ``out_finished`` (uint8 or bool [groups, num_out], may be
    ``finished``) gets each one's parent's entry of ``finished``."""
    dev = logits.device
    if logits.dtype not in _LOGITS_DTYPES:
        raise TypeError(f"logits must be bf16, fp16 or fp32, got {logits.dtype}")
    _need(scores, "scores", torch.float32, dev)
    if scores.dim() != 2:
        raise ValueError("scores must be [groups, beams]")
    G, K = scores.shape
    if logits.dim() == 3 and logits.shape[:2] == (G, K):
        if G > 1 and K > 1 and logits.stride(0) != K * logits.stride(1):
            raise ValueError("the rows of logits must lie at one distance from each other")
        stride = logits.stride(1) if K > 1 else logits.stride(0)
    elif logits.dim() == 2 and logits.shape[0] == G * K:
        stride = logits.stride(0)
    else:
        raise ValueError(f"logits must be [{G * K}, V] or [{G}, {K}, V]")
    V = logits.shape[-1]
    if V > 1 and logits.stride(-1) != 1:
        raise ValueError("the rows of logits must have unit stride")
    if G * K <= 1:
        stride = max(stride, V)
    n = K if num_out is None else int(num_out)
    for t, name, width in ((finished, "finished", K), (out_finished, "out_finished", n)):
        if t is None:
            continue
        if t.dtype not in (torch.uint8, torch.bool):
            raise TypeError(f"{name} must be uint8 or bool, got {t.dtype}")
        _need(t, name, t.dtype, dev)
        if t.shape != (G, width):
            raise ValueError(f"{name} must be [{G}, {width}]")
    if out_finished is not None and out_finished.dtype == torch.bool and finished is not None and finished.dtype != torch.bool:
        raise TypeError("out_finished may be bool only if finished is")
    outs = []
    for t, name, dtype in ((out_scores, "out_scores", torch.float32), (parents, "parents", torch.int32),
                           (tokens, "tokens", torch.int32)):
        if t is None:
            t = torch.empty((G, n), dtype=dtype, device=dev)
        else:
            _need(t, name, dtype, dev)
            if t.shape != (G, n):
                raise ValueError(f"{name} must be [{G}, {n}]")
        outs.append(t)
    if workspace is None:
        workspace = torch.empty(_select_workspace(G, K, V, n), dtype=torch.uint8, device=dev)
    elif workspace.get_device() != logits.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    p = _lib.BeamSelectParams(
        logits.data_ptr(), _LOGITS_DTYPES[logits.dtype], stride, scores.data_ptr(), _ptr(finished), int(pad_token), G, K, V, n,
        outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _ptr(out_finished))
    _call(_lib.load().pa_beam_select, logits, ctypes.byref(p))
    return tuple(outs)


_tensor_device, _element_size, _tensor_shape = torch.Tensor.get_device, torch.Tensor.element_size, operator.attrgetter("shape")


def beam_reorder(parents: torch.Tensor, token_table: torch.Tensor, table_idx: torch.Tensor, seqlens: torch.Tensor,
                 spare_pages: torch.Tensor | None, k_caches, v_caches, *, page_size: int | None = None,
                 prefix_lens: torch.Tensor | None = None, history: torch.Tensor | None = None,
                 max_seqlen_k: int | None = None, kv_dtype: int | None = None) -> None:
    """The paged states follow a selection, in place (``pa_beam_reorder``):
    sequence i of a group becomes the continuation of sequence parents[g, i].
    parents: int32 [groups, beams]; token_table: int32 [rows, width];
    table_idx, seqlens, spare_pages, prefix_lens: int32 [groups * beams], the
    lengths equal within a group; k_caches, v_caches: the pools of every layer
    (lists, or one tensor each), all of one shape, [num_pages, page_size, Hkv, d]
    or, with ``page_size``, [slots, Hkv, d], of 4-bit rows [num_pages, page_size,
    row bytes] or [slots, row bytes]; history: int32 [groups * beams, T].
    ``kv_dtype``, as for ``decode``, tells FP8 from 4-bit pools; without it three
    dimensions of uint8 are 4-bit pages, unless ``page_size`` is given and either
    differs from the second one or the third one is a head size (64 or 128 bytes,
    which no 4-bit row has).
    A moved sequence shares its parent's full pages, and the parent's partly
    filled last page is copied into its spare page; its own last page becomes
    its spare page.  ``spare_pages`` may be None with page size 1.
    ``max_seqlen_k`` (default: the table's width) bounds the lengths."""
    dev = token_table.device
    pools = ([k_caches] if isinstance(k_caches, torch.Tensor) else list(k_caches)) + \
        ([v_caches] if isinstance(v_caches, torch.Tensor) else list(v_caches))
    n = 1 if isinstance(k_caches, torch.Tensor) else len(k_caches)
    if not pools or len(pools) != 2 * n:
        raise ValueError("k_caches and v_caches must hold one pool per layer")
    first = pools[0]
    dtype, shape = first.dtype, first.shape
    # every layer's pools at once (30 us for 32 of them one by one); bits are moved,
    # so that elements of as many bytes are as good as of one type
    if (len(set(map(_tensor_device, pools))) != 1 or not all(map(torch.Tensor.is_contiguous, pools))
            or len(set(map(_element_size, pools))) != 1 or list(map(_tensor_shape, pools)).count(shape) != len(pools)):
        for t in pools:
            _need(t, "every pool", dtype, dev)
        raise ValueError("the pools must have one shape")
    _need(first, "every pool", dtype, dev)
    dims, P = len(shape), page_size
    if not 2 <= dims <= 4:
        raise ValueError("the pools must be [num_pages, page_size, Hkv, d], [slots, Hkv, d] or 4-bit rows")
    paged = dims == 4
    if kv_dtype is not None:
        paged = (_kv_dtype(first, first, kv_dtype) == PA_KV_FP4 and dims == 3) or paged
    elif dims == 3 and dtype == torch.uint8:
        paged = P is None or (P == shape[1] and shape[2] not in (64, 128))
    if paged:
        if P is not None and P != shape[1]:
            raise ValueError("page_size does not match the pool shape")
        num_pages, P = shape[0], shape[1]
    elif P is None:
        raise ValueError("page_size is required for [slots, ...] pools")
    else:
        num_pages = shape[0] // int(P) if int(P) > 0 else 0
    P = int(P)
    row_bytes = math.prod(shape[2 if paged else 1:]) * first.element_size()
    _need(parents, "parents", torch.int32, dev)
    if parents.dim() != 2:
        raise ValueError("parents must be [groups, beams]")
    G, K = parents.shape
    N = G * K
    _need_rows(token_table, "token_table", dev)
    rows, width = token_table.shape
    max_k = width if max_seqlen_k is None else int(max_seqlen_k)
    if max_k > width:
        raise ValueError(f"token_table must be at least {max_k} wide")
    if spare_pages is None and P > 1:
        raise ValueError("spare_pages is required for page sizes over 1")
    for t, name in ((table_idx, "table_idx"), (seqlens, "seqlens"), (spare_pages, "spare_pages"), (prefix_lens, "prefix_lens")):
        if t is not None:
            _need(t, name, torch.int32, dev)
            if t.numel() != N:
                raise ValueError(f"{name} must hold one entry per sequence ({N})")
    history_ptr, history_stride, history_len = None, 0, 0
    if history is not None:
        _need_rows(history, "history", dev)
        if history.shape[0] != G * K:
            raise ValueError(f"history must have a row per sequence ({G * K})")
        if history.numel():
            history_ptr, history_len = history.data_ptr(), history.shape[1]
            history_stride = max(history.stride(0), history_len)
    ptrs = array.array("Q", map(torch.Tensor.data_ptr, pools))
    p = _lib.BeamReorderParams(
        parents.data_ptr(), G, K, P, max_k, token_table.data_ptr(), max(token_table.stride(0), width), rows, table_idx.data_ptr(),
        seqlens.data_ptr(), _ptr(prefix_lens), _ptr(spare_pages), ptrs.buffer_info()[0], len(pools), num_pages, row_bytes,
        history_ptr, history_stride, history_len)
    _call(_lib.load().pa_beam_reorder, token_table, ctypes.byref(p))
