"""Malformed calls of the shared-prefix decode and of beam search that libpa must reject on the host, before any
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

DEC = dict(q=0x1000, k_cache=0x2000, v_cache=0x3000, page_table=0x4000, page_table_stride=64, cache_seqlens=0x5000, num_seqs=8,
           max_seqlen_k=1000, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=100, scale=0.125, out=0x6000,
           lse=None, workspace=0x10000, workspace_bytes=1 << 40, kv_chunk=0, kv_dtype=0, k_scale=None, v_scale=None,
           sliding_window=0, max_ctas=0, overlap_previous=0)
SHARED = dict(cu_groups=0x7000, prefix_lens=0x8000, num_groups=2, max_group=8, max_prefix=900, max_suffix=200)
SHARED_CASES = [
    ("negative_groups", dict(num_groups=-1), INVALID),
    ("negative_prefix", dict(max_prefix=-1), INVALID),
    ("group_over_batch", dict(max_group=9), INVALID),
    ("prefix_over_length", dict(max_prefix=1001), INVALID),
    ("suffix_over_length", dict(max_suffix=1001), INVALID),
    ("window", dict(sliding_window=64), UNSUPPORTED),
    ("max_ctas", dict(max_ctas=3), UNSUPPORTED),
    ("overlap", dict(overlap_previous=1), UNSUPPORTED),
    ("too_many_groups", dict(num_groups=16385), UNSUPPORTED),
    ("too_many_steps", dict(num_groups=16384, num_seqs=8192, max_group=8192, max_prefix=60000, max_seqlen_k=60000, max_suffix=1,
                            page_table_stride=4000), UNSUPPORTED),
    ("null_groups", dict(cu_groups=None), INVALID),
    ("null_prefixes", dict(prefix_lens=None), INVALID),
    ("null_q", dict(q=None), INVALID),
    ("misaligned_q", dict(q=0x1008), INVALID),
    ("misaligned_workspace", dict(workspace=0x10008), INVALID),
    ("small_workspace", dict(workspace_bytes=1000), INVALID),
    ("no_workspace", dict(workspace=None), INVALID),
    ("narrow_table", dict(page_table_stride=62), INVALID),
    ("head_dim96", dict(head_dim=96), UNSUPPORTED),
    ("group3", dict(num_q_heads=6), UNSUPPORTED),
    ("page8", dict(page_size=8), UNSUPPORTED),
    ("scale0", dict(scale=0.0), INVALID),
    ("fp8_no_scales", dict(kv_dtype=1), INVALID),
    ("fp4_no_scales", dict(kv_dtype=2), INVALID),
    ("empty_batch", dict(num_seqs=0, max_group=0, q=None, out=None, workspace=None, cu_groups=None), OK),
]
SELECT = dict(logits=0x1000, logits_dtype=0, logits_stride=1000, scores=0x2000, finished=None, pad_token=0, num_groups=2, beams=4,
              vocab=1000, num_out=4, out_scores=0x3000, out_parents=0x4000, out_tokens=0x5000, workspace=0x6000,
              workspace_bytes=1 << 40)
SELECT_CASES = [
    ("negative_groups", dict(num_groups=-1), INVALID),
    ("no_beams", dict(beams=0), UNSUPPORTED),
    ("beams65", dict(beams=65), UNSUPPORTED),
    ("no_vocab", dict(vocab=0), UNSUPPORTED),
    ("vocab2_24", dict(vocab=1 << 24, logits_stride=1 << 24), UNSUPPORTED),
    ("out0", dict(num_out=0), UNSUPPORTED),
    ("out129", dict(num_out=129), UNSUPPORTED),
    ("out_over_vocab", dict(vocab=3), UNSUPPORTED),
    ("too_many_rows", dict(num_groups=16384), UNSUPPORTED),
    ("dtype3", dict(logits_dtype=3), INVALID),
    ("stride", dict(logits_stride=999), INVALID),
    ("pad", dict(pad_token=1000), INVALID),
    ("negative_pad", dict(pad_token=-1), INVALID),
    ("null_logits", dict(logits=None), INVALID),
    ("null_scores", dict(scores=None), INVALID),
    ("null_out", dict(out_tokens=None), INVALID),
    ("misaligned", dict(logits=0x1002), INVALID),
    ("small_workspace", dict(workspace_bytes=100), INVALID),
    ("no_workspace", dict(workspace=None), INVALID),
    ("misaligned_workspace", dict(workspace=0x6008), INVALID),
    ("in_place_other_size", dict(out_scores=0x2000, num_out=5), INVALID),
    ("no_groups", dict(num_groups=0, logits=None, scores=None, workspace=None), OK),
]
REORDER = dict(parents=0x1000, num_groups=2, beams=4, page_size=16, max_seqlen_k=100, token_table=0x2000, token_table_stride=128,
               token_table_rows=8, table_idx=0x3000, seqlens=0x4000, prefix_lens=None, spare_pages=0x5000, num_pools=2,
               num_pages=100, row_bytes=256, history=None, history_stride=0, history_len=0)
REORDER_CASES = [
    ("negative_groups", dict(num_groups=-1), INVALID),
    ("beams65", dict(beams=65), UNSUPPORTED),
    ("page8", dict(page_size=8), UNSUPPORTED),
    ("narrow_table", dict(token_table_stride=99), INVALID),
    ("row24", dict(row_bytes=24), UNSUPPORTED),
    ("row0", dict(row_bytes=0), UNSUPPORTED),
    ("too_many_pools", dict(num_pools=257), UNSUPPORTED),
    ("too_many_pages", dict(num_pages=1 << 28), UNSUPPORTED),
    ("too_many_rows", dict(num_groups=16384), UNSUPPORTED),
    ("null_parents", dict(parents=None), INVALID),
    ("null_spares", dict(spare_pages=None), INVALID),
    ("null_pool", dict(pools=[0x10000, 0]), INVALID),
    ("misaligned_pool", dict(pools=[0x10000, 0x20008]), INVALID),
    ("narrow_history", dict(history=0x8000, history_stride=9, history_len=10), INVALID),
    ("negative_history", dict(history_len=-1), INVALID),
    ("no_groups", dict(num_groups=0, parents=None, token_table=None), OK),
]


def expected():
    out = {}
    for name, cases in (("shared", SHARED_CASES), ("select", SELECT_CASES), ("reorder", REORDER_CASES)):
        out.update({f"{name}-{c}": want for c, _, want in cases})
    return out


def main():
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    out = {}

    def note(case, status):
        out[case] = [int(status), lib.pa_last_error().decode()]

    for c, change, _ in SHARED_CASES:
        dec = {**DEC, **{k: v for k, v in change.items() if k in DEC}}
        rest = {**SHARED, **{k: v for k, v in change.items() if k in SHARED}}
        p = _lib.DecodeSharedParams(dec=_lib.DecodeParams(**dec), **rest)
        note(f"shared-{c}", lib.pa_decode_shared(ctypes.byref(p), None))
    for c, change, _ in SELECT_CASES:
        note(f"select-{c}", lib.pa_beam_select(ctypes.byref(_lib.BeamSelectParams(**{**SELECT, **change})), None))
    for c, change, _ in REORDER_CASES:
        args = {**REORDER, **change}
        pools = args.pop("pools", [0x10000, 0x20000])
        arr = (ctypes.c_void_p * 300)(*pools)
        note(f"reorder-{c}", lib.pa_beam_reorder(ctypes.byref(_lib.BeamReorderParams(pools=ctypes.addressof(arr), **args)), None))
    for name, fn in (("shared", lib.pa_decode_shared), ("select", lib.pa_beam_select), ("reorder", lib.pa_beam_reorder)):
        assert fn(None, None) == INVALID, name
    print(json.dumps(out))


if __name__ == "__main__":
    main()
