"""Device data of decode over shared prefixes that the error word tells of, and data that
it must not."""
import pytest
import torch

from test_shared_decode_gpu import FP4, FP8, check, make, reference

pytestmark = pytest.mark.gpu


def call(s, **kw):
    import paged_kv_flashattention_gb300 as pa
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    out = pa.decode_shared(s["q"], *s["pools"], s["table"], s["lens"], s["max_k"], s["cu"], s["first"], lse=lse,
                           **{**s["bounds"], "max_suffix": s["max_k"], **s["scales"], **kw})
    return (out, lse), pa.device_error()


@pytest.mark.parametrize("kv", [0, FP8, FP4])
@pytest.mark.parametrize("which", [[1], [2], [1, 2], [3], [4, 5], [1, 3]])
def test_no_prefix_in_a_group_that_has_one(cuda_device, which, kv):
    """A prefix that differs from its group's, though it is none.  (The sequences without are
    right, through their own rows; where the first one has none its group has none.)"""
    import paged_kv_flashattention_gb300 as pa
    s = make(cuda_device, 5, [3, 3], [200, 96], [5, 6, 7, 8, 9, 10, 11], 8, 2, 64, 16, kv, loose=1)
    s["ref"] = reference(s)
    s["first"][which] = 0
    got, bits = call(s)
    assert bits & pa.PA_DEVERR_SEQLENS
    lost = [4, 5] if 3 in which else []                  # a prefix, in a group without
    check(s, got, rows=[b for b in range(7) if b not in lost])


@pytest.mark.parametrize("kv", [0, FP4])
def test_quiet(cuda_device, kv):
    """Groups without a prefix, padding rows with and without one, sequences of no group, and
    groups of padding rows alone: nothing to tell."""
    s = make(cuda_device, 6, [3, 2, 4, 2], [200, 0, 64, 48], [5, 6, 7, 8, 9, 10, 11, 3, 3, 1, 1, 20, 0], 8, 2, 64, 16, kv, loose=2)
    for b, keep in ((1, False), (6, True), (9, True), (10, False), (12, False)):
        s["lens"][b] = 0
        s["host"][0][b] = 0
        if not keep:
            s["first"][b] = 0
    got, bits = call(s)
    assert bits == 0
    check(s, got)
