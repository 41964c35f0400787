"""Paged-KV exact attention for GB300 (sm_103a).

A small C-ABI library (``libpa.so``, declared in ``include/pa.h``) with
hand-written CUDA kernels for the KV-cache store (bf16, FP8 E4M3 with
per-head scales, or 4-bit rows with block scales), the batch's metadata, varlen causal prefill / extend attention over a page table,
split-KV decode and the log-sum-exp combine, both attention halves of a mixed
batch in one launch, decode over prefixes that sequences share, and beam
search's selection and reordering; this package is its thin torch binding.  PyTorch
provides device memory and streams only.
"""
from .api import (PA_DEVERR_NO_PAGES, PA_DEVERR_PAGE_RANGE, PA_DEVERR_POSITION, PA_DEVERR_SEQLENS, PA_DEVERR_TABLE_INDEX,
                  PA_DEVERR_TIMEOUT, PA_KV_BF16, PA_KV_FP4, PA_KV_FP8_E4M3, PA_MIXED_SCHEDULER_INTS, PagedAttentionError,
                  abi_version, beam_reorder, beam_select, beam_select_workspace_size,
                  build_batch, build_page_table,
                  build_seqlens, decode, decode_noalloc, decode_kv_chunk, decode_shared, decode_shared_workspace_size,
                  decode_workspace_size,
                  device_error, fp4_row_bytes, load_kv_fp4, lse_combine, mixed_batch, prefill, prefill_scheduler, rope_cos_sin_table,
                  rope_store_kv, store_kv, store_kv_fp4, store_kv_fp8)

from .beams import BeamSearch
from .graphs import DecodeGraphRunner, bucket_for
from .metadata import BatchPlanner

__all__ = [
    "PagedAttentionError", "abi_version", "build_batch", "BatchPlanner", "build_page_table", "build_seqlens", "decode",
    "decode_noalloc", "decode_shared", "decode_shared_workspace_size", "beam_select", "beam_select_workspace_size",
    "beam_reorder", "BeamSearch",
    "decode_kv_chunk", "decode_workspace_size", "device_error", "lse_combine", "mixed_batch", "prefill",
    "prefill_scheduler",
    "DecodeGraphRunner", "bucket_for",
    "store_kv", "store_kv_fp8", "store_kv_fp4", "load_kv_fp4", "fp4_row_bytes",
    "PA_KV_BF16", "PA_KV_FP8_E4M3", "PA_KV_FP4", "PA_MIXED_SCHEDULER_INTS",
    "rope_cos_sin_table", "rope_store_kv",
    "PA_DEVERR_PAGE_RANGE", "PA_DEVERR_SEQLENS", "PA_DEVERR_TIMEOUT", "PA_DEVERR_POSITION",
    "PA_DEVERR_TABLE_INDEX", "PA_DEVERR_NO_PAGES",
]
