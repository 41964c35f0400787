"""What 4-bit decodes need of a workspace and what the library reports, read
from its host checks: a call whose workspace holds one byte is refused with the
size it needs (the pointers are made up, nothing is launched)."""
from __future__ import annotations

import ctypes
import re

import fp4_reject_cases as R


def _params(n, keys, hq, hkv, d, window, chunk, **kw):
    from paged_kv_flashattention_gb300 import _lib
    return _lib.DecodeParams(**{**R.DECODE, "num_seqs": n, "max_seqlen_k": keys, "num_q_heads": hq, "num_kv_heads": hkv,
                                "head_dim": d, "page_table_stride": keys // 16 + 1, "num_pages": 1 << 20,
                                "sliding_window": window, "kv_chunk": chunk, **kw})


def needed(n, keys, hq, hkv, d, window=0, chunk=0):
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    p = _params(n, keys, hq, hkv, d, window, chunk, workspace_bytes=1)
    assert lib.pa_decode(ctypes.byref(p), None) == R.INVALID
    return int(re.search(r"workspace of (\d+) bytes needed", lib.pa_last_error().decode()).group(1))


def reported(n, keys, hq, hkv, d, window=0, chunk=0):
    from paged_kv_flashattention_gb300 import _lib
    p = _params(n, keys, hq, hkv, d, window, chunk)
    return int(_lib.load().pa_decode_workspace_size(ctypes.byref(p)))


KEYS = (0, 1, 63, 64, 65, 700, 2047, 2048, 2049, 4096, 6080, 8192, 9728, 10033, 12160, 19456, 20011, 32768, 131072)
HEADS = ((32, 8, 128), (32, 8, 64), (4, 1, 64), (64, 16, 64), (24, 12, 128), (15, 15, 128), (64, 64, 64))


def check_smaller_batches():
    """The size reported for N sequences holds every n <= N."""
    for hq, hkv, d in HEADS:
        for keys in KEYS:
            for window in (0, 15, 700, 5000):
                most, last = 0, 0
                for n in (*range(1, 33), 100, 151, 152, 153, 512):
                    most = max(most, needed(n, keys, hq, hkv, d, window))
                    size = reported(n, keys, hq, hkv, d, window)
                    assert size >= most, f"{n} x {keys} {hq}/{hkv} d{d} window {window}: {size} < {most}"
                    assert size >= last, f"{n} x {keys} {hq}/{hkv} d{d} window {window}: smaller than for fewer"
                    last = size


def check_shorter_bounds_and_windows():
    """The size reported without a window holds any window, and any smaller
    max_seqlen_k."""
    for hq, hkv, d in HEADS:
        for n in (1, 2, 3, 5, 8, 200):
            most = 0
            for keys in KEYS:
                for window in (0, 1, 15, 16, 17, 333, 5000):
                    most = max(most, needed(n, keys, hq, hkv, d, window))
                size = reported(n, keys, hq, hkv, d)
                assert size >= most, f"{n} x {keys} {hq}/{hkv} d{d}: {size} < {most}"


def check_not_wasteful():
    """It stays within what the largest batch needs and a GPU's worth of ranges
    more: 157 slots a KV-head group (152 SMs), and three a sequence."""
    for hq, hkv, d in HEADS:
        for keys in KEYS:
            for n in (1, 2, 4, 8, 64, 256):
                extra = (160 + 3 * n) * hq * (d * 4 + 4) + 1024
                assert reported(n, keys, hq, hkv, d) <= needed(n, keys, hq, hkv, d) + extra


def check_given_ranges():
    """With the caller's kv_chunk the size is the need itself."""
    for n in (1, 3, 40):
        for keys in KEYS:
            assert reported(n, keys, 32, 8, 128, 0, 64) == needed(n, keys, 32, 8, 128, 0, 64)
