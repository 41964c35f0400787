"""Malformed calls of the 4-bit entry points and the batch plan that libpa must reject on the host, before any
launch; run as a script with no GPU visible (the pointers are made up), it
prints one JSON object {case id: [status, last error]}."""
from __future__ import annotations

import ctypes
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

OK, INVALID, UNSUPPORTED = 0, 1, 2

# k, v, slots, tokens, k_cache, v_cache, slots, hkv, d, k_scale, v_scale, stream
STORE = (0x1000, 0x2000, 0x3000, 4, 0x4000, 0x5000, 64, 2, 64, 0x6000, 0x7000, None)
STORE_CASES = [
    ("misaligned_k", {0: 0x1008}, INVALID),
    ("misaligned_pool", {4: 0x4001}, INVALID),
    ("null_scale", {9: None}, INVALID),
    ("null_slots", {2: None}, INVALID),
    ("negative_tokens", {3: -1}, INVALID),
    ("negative_slots", {6: -1}, INVALID),
    ("head_dim96", {8: 96}, UNSUPPORTED),
    ("no_heads", {7: 0}, INVALID),
    ("row_too_long", {7: 64, 8: 128}, UNSUPPORTED),
    ("too_many_tokens", {3: 1 << 31}, UNSUPPORTED),
    ("zero_tokens", {0: None, 1: None, 2: None, 3: 0, 4: None, 5: None, 9: None, 10: None}, OK),
]
ROPE = dict(q=0x1000, q_out=0x1000, k=0x2000, v=0x3000, positions=0x4000, cos_sin=0x5000, max_pos=64, rot_dim=64,
            interleaved=0, slot_mapping=0x6000, num_tokens=4, num_q_heads=8, num_kv_heads=2, head_dim=64, k_cache=0x7000,
            v_cache=0x8000, num_slots=64, kv_dtype=2, k_scale=0x9000, v_scale=0x9100)
ROPE_CASES = [
    ("no_scales", dict(k_scale=None), INVALID),
    ("head_dim32", dict(head_dim=32, rot_dim=32), UNSUPPORTED),
    ("kv_dtype3", dict(kv_dtype=3), INVALID),
    ("misaligned_pool", dict(v_cache=0x8008), INVALID),
]

DECODE = dict(q=0x1000, k_cache=0x2000, v_cache=0x3000, page_table=0x4000, page_table_stride=64, cache_seqlens=0x5000,
              num_seqs=2, max_seqlen_k=512, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=1000,
              scale=0.1, out=0x7000, lse=None, workspace=0x8000, workspace_bytes=1 << 30, kv_chunk=0, kv_dtype=2,
              k_scale=0x9000, v_scale=0x9100)
DECODE_CASES = [
    ("no_scales", dict(k_scale=None), INVALID),
    ("head_dim96", dict(head_dim=96), UNSUPPORTED),
    ("page8", dict(page_size=8), UNSUPPORTED),
    ("group3", dict(num_q_heads=6), UNSUPPORTED),
    ("small_workspace", dict(workspace_bytes=4096), INVALID),
    ("misaligned_pool", dict(k_cache=0x2008), INVALID),
    ("table_stride", dict(page_table_stride=31), INVALID),
    ("scale_zero", dict(scale=0.0), INVALID),
    ("keys_overflow_int32", dict(num_seqs=16384, max_seqlen_k=1 << 18, page_table_stride=1 << 14, num_pages=1 << 20,
                                 kv_chunk=1 << 16), UNSUPPORTED),
    ("no_sequences", dict(num_seqs=0), OK),
]
PREFILL = dict(q=0x1000, k_cache=0x2000, v_cache=0x3000, page_table=0x4000, page_table_stride=64, total_q=100,
               cu_seqlens_q=0x5000, cu_seqlens_k=0x6000, num_seqs=2, max_seqlen_q=64, max_seqlen_k=512, num_q_heads=8,
               num_kv_heads=2, head_dim=128, page_size=16, num_pages=1000, causal=1, scale=0.1, out=0x7000, lse=None,
               lse_stride=0, kv_dtype=2, k_scale=0x9000, v_scale=0x9100, scheduler=0xA000)
PREFILL_CASES = [
    ("no_scales", dict(v_scale=None), INVALID),
    ("kv_dtype3", dict(kv_dtype=3), INVALID),
    ("head_dim32", dict(head_dim=32), UNSUPPORTED),
    ("page8", dict(page_size=8), UNSUPPORTED),
    ("group3", dict(num_q_heads=6), UNSUPPORTED),
    ("misaligned_pool", dict(k_cache=0x2008), INVALID),
    ("table_stride", dict(page_table_stride=31), INVALID),
    ("scale_zero", dict(scale=0.0), INVALID),
    ("no_scheduler", dict(scheduler=None), INVALID),
    ("no_tokens", dict(total_q=0), OK),
]
# One launch for prefill and decode takes bf16 and FP8 pools only.
MIXED_CASES = [
    ("both_4bit", {}, {}, UNSUPPORTED),
    ("prefill_4bit", {}, dict(kv_dtype=1), UNSUPPORTED),
    ("decode_4bit", dict(kv_dtype=1), {}, UNSUPPORTED),
]
BATCH = dict(cached_len=0x1000, extend_len=0x2000, num_seqs=4, max_seqlen_k=100, page_size=16, token_table=0x3000,
             token_table_stride=100, token_table_rows=8, table_idx=0x4000, free_pages=0x5000, num_free_pages=8, num_tokens=40,
             cu_seqlens_q=0x6000, cu_seqlens_k=0x7000, cache_seqlens=0x8000, positions=0x9000, slot_mapping=0xA000,
             page_table=0xB000, page_table_stride=7, totals=0xC000)
BATCH_CASES = [
    ("negative_seqs", dict(num_seqs=-1), INVALID),
    ("negative_tokens", dict(num_tokens=-1), INVALID),
    ("negative_free", dict(num_free_pages=-1), INVALID),
    ("page0", dict(page_size=0), INVALID),
    ("too_many_seqs", dict(num_seqs=16385), UNSUPPORTED),
    ("keys_overflow_int32", dict(num_seqs=16384, max_seqlen_k=1 << 17, token_table_stride=1 << 17,
                                 page_table_stride=1 << 13), UNSUPPORTED),
    ("too_many_tokens", dict(num_tokens=1 << 31), UNSUPPORTED),
    ("page_table_stride", dict(page_table_stride=6), INVALID),
    ("token_table_stride", dict(token_table_stride=99), INVALID),
    ("null_lens", dict(extend_len=None), INVALID),
    ("null_slots", dict(slot_mapping=None), INVALID),
    ("null_totals", dict(totals=None), INVALID),
]


def expected():
    out = {f"store/{i}": s for i, _, s in STORE_CASES}
    out.update({f"load/{i}": s for i, _, s in STORE_CASES})
    out.update({f"rope/{i}": s for i, _, s in ROPE_CASES})
    out.update({f"decode/{i}": s for i, _, s in DECODE_CASES})
    out.update({f"prefill/{i}": s for i, _, s in PREFILL_CASES})
    out.update({f"mixed/{i}": s for i, _, _, s in MIXED_CASES})
    out.update({f"batch/{i}": s for i, _, s in BATCH_CASES})
    return out


def run_all() -> dict:
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    res = {}

    def rec(key, status):
        res[key] = [int(status), lib.pa_last_error().decode(errors="replace")]

    for i, change, _ in STORE_CASES:
        a = [change.get(n, x) for n, x in enumerate(STORE)]
        rec(f"store/{i}", lib.pa_store_kv_fp4(*a))
        # slots, tokens, k_cache, v_cache, slots, hkv, d, scales, k_out, v_out, stream
        rec(f"load/{i}", lib.pa_load_kv_fp4(a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[0], a[1], None))
    for i, kw, _ in ROPE_CASES:
        p = _lib.RopeStoreParams(**{**ROPE, **kw})
        rec(f"rope/{i}", lib.pa_rope_store_kv(ctypes.byref(p), None))
    for i, kw, _ in DECODE_CASES:
        p = _lib.DecodeParams(**{**DECODE, **kw})
        rec(f"decode/{i}", lib.pa_decode(ctypes.byref(p), None))
    for i, kw, _ in PREFILL_CASES:
        p = _lib.PrefillParams(**{**PREFILL, **kw})
        rec(f"prefill/{i}", lib.pa_prefill(ctypes.byref(p), None))
    for i, kp, kd, _ in MIXED_CASES:
        p, d = _lib.PrefillParams(**{**PREFILL, **kp}), _lib.DecodeParams(**{**DECODE, **kd})
        rec(f"mixed/{i}", lib.pa_mixed_batch(ctypes.byref(p), ctypes.byref(d), None))
    for i, kw, _ in BATCH_CASES:
        p = _lib.BatchParams(**{**BATCH, **kw})
        rec(f"batch/{i}", lib.pa_build_batch(ctypes.byref(p), None))
    return res


if __name__ == "__main__":
    print(json.dumps(run_all()))
