"""Refusals of selection's ``out_finished`` on the host."""
import ctypes

import pytest
import torch

import beam_reject_cases


def test_in_place_needs_as_many():
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    p = _lib.BeamSelectParams(**{**beam_reject_cases.SELECT, "num_out": 5, "finished": 0x9000, "out_finished": 0x9000})
    assert lib.pa_beam_select(ctypes.byref(p), None) == beam_reject_cases.INVALID
    assert b"out_finished" in lib.pa_last_error()


def test_binding():
    import paged_kv_flashattention_gb300 as pa
    x, s = torch.zeros((8, 50)), torch.zeros((2, 4))
    flags = lambda *shape, dtype=torch.uint8: torch.zeros(shape, dtype=dtype)
    for kw in (dict(out_finished=flags(2, 3)), dict(num_out=5, out_finished=flags(2, 4)), dict(out_finished=flags(8)),
               dict(out_finished=flags(4, 2).t())):
        with pytest.raises(ValueError):
            pa.beam_select(x, s, **kw)
    for kw in (dict(out_finished=flags(2, 4, dtype=torch.int32)), dict(finished=flags(2, 4), out_finished=flags(2, 4, dtype=torch.bool))):
        with pytest.raises(TypeError):
            pa.beam_select(x, s, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        pa.beam_select(x, s, finished=flags(2, 4), out_finished=flags(2, 4))
