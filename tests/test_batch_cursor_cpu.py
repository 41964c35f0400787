"""Refusals of the batch plan's cursor, on the host."""
import pytest
import torch


def test_binding_checks():
    import paged_kv_flashattention_gb300 as pa
    pl = pa.BatchPlanner("cpu", 4, 16, 100, 16)
    c = torch.zeros(3, dtype=torch.int32)
    tt, idx, free = torch.zeros((5, 100), dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="needs free_pages"):
        pl.build(c, c, tt, idx, free_cursor=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="2 int32"):
        pl.build(c, c, tt, idx, free_pages=free, free_cursor=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        pl.build(c, c, tt, idx, free_pages=free, free_cursor=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        pl.build(c, c, tt, idx, free_pages=free, free_cursor=torch.zeros((2, 2), dtype=torch.int32)[:, 0])


def test_cursor_without_a_list():
    """The C call refuses it before any launch (made-up pointers)."""
    import ctypes
    import fp4_reject_cases
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    p = _lib.BatchParams(**{**fp4_reject_cases.BATCH, "free_pages": None})
    assert lib.pa_build_batch_from(ctypes.byref(p), 0xD000, None) == fp4_reject_cases.INVALID
    assert b"free_pages" in lib.pa_last_error()
