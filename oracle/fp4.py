"""Oracle of the 4-bit KV cache (numpy, fp64): the row format, its store and
read-back, and attention over 4-bit pools.

TEST INFRASTRUCTURE ONLY, like the rest of the package: nothing is shared with
the library.  Everything is written from the format's definition in
``include/pa.h``: codes are found by searching a table of the values, single
rounding to fp32 happens where the format names an IEEE single operation, and
the rest is double precision.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# E4M3 magnitudes by code 0 .. 126 (127 is NaN)
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])


def layout(hkv: int, d: int):
    """(heads of a group, groups, code bytes of a group, group bytes, row bytes)."""
    gs = max(p for p in (1, 2, 4, 8) if hkv % p == 0)
    code = gs * d // 2
    group = code + gs * d // 16
    group += -group % 16
    return gs, hkv // gs, code, group, group * (hkv // gs)


def nearest_code(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table's entry nearest to each x >= 0, ties to the even
    index, x beyond the table to its end."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        dlo, dhi = x - table[lo], table[hi] - x
    code = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(x >= table[-1], len(table) - 1, code)


def quantise(x: np.ndarray, head_scale: np.ndarray):
    """x float [T, Hkv, d] to (codes 0..15 uint8 [T, Hkv, d], scale codes uint8
    [T, Hkv, d/16])."""
    T, hkv, d = x.shape
    x = np.asarray(x, np.float32).reshape(T, hkv, d // 16, 16)
    g = np.asarray(head_scale, np.float32)[None, :, None]
    nan = np.isnan(x).any(-1)
    with np.errstate(all="ignore"):
        amax = np.where(nan, np.float32(0), np.nan_to_num(np.abs(x), nan=0.0, posinf=np.inf).max(-1))
        want = ((amax / g).astype(np.float32) / np.float32(6)).astype(np.float32)
        sc = nearest_code(want, E4M3)
        step = (E4M3[sc].astype(np.float32) * g).astype(np.float32)[..., None]
        z = np.where(step > 0, (x / step).astype(np.float32), np.float32(0))
        z = np.where(nan[..., None], np.float32(0), z)
    code = nearest_code(np.abs(z), E2M1) + 8 * (np.signbit(z) & (step > 0) & ~nan[..., None])
    return code.astype(np.uint8).reshape(T, hkv, d), np.where(nan, 127, sc).astype(np.uint8)


def pack(codes: np.ndarray, scales: np.ndarray, rows: np.ndarray | None = None) -> np.ndarray:
    """Codes and scale codes to pool rows uint8 [T, row bytes]; the padding
    keeps what ``rows`` held."""
    T, hkv, d = codes.shape
    gs, groups, cb, gb, rb = layout(hkv, d)
    out = np.zeros((T, rb), np.uint8) if rows is None else rows.copy()
    for h in range(hkv):
        base, i = (h // gs) * gb, h % gs
        out[:, base + i * d // 2:base + (i + 1) * d // 2] = codes[:, h, 0::2] + 16 * codes[:, h, 1::2]
        out[:, base + cb + i * d // 16:base + cb + (i + 1) * d // 16] = scales[:, h]
    return out


def unpack(rows: np.ndarray, hkv: int, d: int, head_scale) -> np.ndarray:
    """Pool rows [..., row bytes] to the float64 values [..., Hkv, d]."""
    gs, groups, cb, gb, rb = layout(hkv, d)
    assert rows.shape[-1] == rb
    lead = rows.shape[:-1]
    r = rows.reshape(-1, rb)
    signed = np.concatenate([E2M1, -E2M1])
    scale_of = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    out = np.empty((r.shape[0], hkv, d))
    for h in range(hkv):
        base, i = (h // gs) * gb, h % gs
        b = r[:, base + i * d // 2:base + (i + 1) * d // 2]
        out[:, h, 0::2] = signed[b % 16]
        out[:, h, 1::2] = signed[b // 16]
        s = scale_of[r[:, base + cb + i * d // 16:base + cb + (i + 1) * d // 16]]
        out[:, h] *= np.repeat(s, 16, axis=1) * float(head_scale[h])
    return out.reshape(*lead, hkv, d)


def store(x, slots, pool_rows: np.ndarray, head_scale) -> None:
    """Write x float [T, Hkv, d] to pool_rows uint8 [slots, row bytes] in place;
    negative slots are skipped."""
    codes, scales = quantise(x, head_scale)
    live = np.asarray(slots) >= 0
    at = np.asarray(slots)[live]
    pool_rows[at] = pack(codes[live], scales[live], pool_rows[at])


def attention(q, k_rows, v_rows, page_table, cu_q, cu_k, *, num_kv_heads: int, page_size: int, k_scale, v_scale,
              scale: float, causal: bool = True, window: int = 0, block_mask=None):
    """Attention over 4-bit pools in fp64: q float [total_q, Hq, d]; k_rows,
    v_rows uint8 [slots, row bytes].  Returns (out [total_q, Hq, d], lse
    [total_q, Hq], mag [total_q, Hq, d]); mag is the attention over |V|, the
    yardstick of rounding errors in P.  Rows that see no key give 0, -inf, 0."""
    total, hq, d = q.shape
    G = hq // num_kv_heads
    out, mag = np.zeros((total, hq, d)), np.zeros((total, hq, d))
    lse = np.full((total, hq), -np.inf)
    for b in range(len(cu_q) - 1):
        lq, lk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        if lq == 0 or lk == 0:
            continue
        j = np.arange(lk)
        slot = np.asarray(page_table[b])[j // page_size].astype(np.int64) * page_size + j % page_size
        k = unpack(k_rows[slot], num_kv_heads, d, k_scale)
        v = unpack(v_rows[slot], num_kv_heads, d, v_scale)
        i = np.arange(lq)[:, None]
        pos = lk - lq + i
        see = np.ones((lq, lk), bool)
        if causal:
            see &= j[None] <= pos
        if window > 0:
            see &= j[None] >= pos - (window - 1)
        if block_mask is not None:
            see &= np.asarray(block_mask[b])[i // 128, j[None] // 128] != 0
        for h in range(hq):
            s = q[cu_q[b]:cu_q[b + 1], h].astype(np.float64) @ k[:, h // G].T * scale
            s = np.where(see, s, -np.inf)
            m = s.max(1)
            some = m > -np.inf
            p = np.exp(s - np.where(some, m, 0.0)[:, None])
            l = p.sum(1)
            rows = slice(int(cu_q[b]), int(cu_q[b + 1]))
            p = np.where(some[:, None], p, 0.0)
            out[rows, h] = (p @ v[:, h // G]) / np.where(some, l, 1.0)[:, None]
            mag[rows, h] = (p @ np.abs(v[:, h // G])) / np.where(some, l, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                lse[rows, h] = np.where(some, m + np.log(np.where(some, l, 1.0)), -np.inf)
    return out, lse, mag
