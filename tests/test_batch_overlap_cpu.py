"""The batch plan reads its lengths, rows and free list in every CTA while it
writes its outputs: an input that lies on an output is refused on the host,
before any launch (the pointers are made up)."""
import ctypes

import pytest

import fp4_reject_cases as R

B, T = 4, 40
OUT = {"cu_seqlens_q": B + 1, "cu_seqlens_k": B + 1, "cache_seqlens": B, "positions": T, "slot_mapping": T, "totals": 4}
IN = {"cached_len": B, "extend_len": B, "table_idx": B, "free_pages": 8}


def status(cursor=None, **kw):
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    p = _lib.BatchParams(**{**R.BATCH, **kw})
    assert (p.num_seqs, p.num_tokens, p.num_free_pages) == (B, T, 8)
    return lib.pa_build_batch_from(ctypes.byref(p), cursor, None), lib.pa_last_error().decode()


@pytest.mark.parametrize("out", sorted(OUT))
@pytest.mark.parametrize("name", sorted(IN))
def test_inputs_on_outputs(name, out):
    at, n = R.BATCH[out], OUT[out]
    for where in (at, at + 4 * (n - 1), at - 4 * (IN[name] - 1)):      # the same start, last entry, first entry
        st, msg = status(**{name: where})
        assert st == R.INVALID and name in msg and "overlaps" in msg


@pytest.mark.parametrize("out", sorted(OUT))
def test_cursor_on_outputs(out):
    for where in (R.BATCH[out] - 4, R.BATCH[out] + 4 * (OUT[out] - 1)):
        st, msg = status(cursor=where)
        assert st == R.INVALID and "free_cursor overlaps" in msg


@pytest.mark.parametrize("name", sorted(IN))
def test_cursor_on_inputs(name):
    st, msg = status(cursor=R.BATCH[name] + 4 * (IN[name] - 1))
    assert st == R.INVALID and f"{name} overlaps" in msg
