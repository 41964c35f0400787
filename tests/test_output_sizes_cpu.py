"""Outputs that are too small for a call are refused by the binding before any
launch (CPU tensors, so nothing could be launched either way)."""
import pytest
import torch


def pools(fp4, hkv=2, d=64):
    import paged_kv_flashattention_gb300 as pa
    if fp4:
        return [torch.zeros((4, 16, pa.fp4_row_bytes(hkv, d)), dtype=torch.uint8) for _ in range(2)]
    return [torch.zeros((4, 16, hkv, d), dtype=torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("fp4", [False, True])
def test_rotated_q(fp4):
    import paged_kv_flashattention_gb300 as pa
    T, hq, hkv, d = 3, 8, 2, 64
    q, k = torch.zeros((T, hq, d), dtype=torch.bfloat16), torch.zeros((T, hkv, d), dtype=torch.bfloat16)
    i, cs, g = torch.zeros(T, dtype=torch.int32), torch.zeros((16, d)), torch.ones(hkv)
    kw = dict(k_scale=g, v_scale=g, kv_dtype=pa.PA_KV_FP4) if fp4 else {}
    for small in (q[:2], torch.zeros((T, hq, d - 16), dtype=torch.bfloat16), q[:0]):
        with pytest.raises(ValueError, match="q_out"):
            pa.rope_store_kv(q, k, k, i, cs, i, *pools(fp4), q_out=small, **kw)


@pytest.mark.parametrize("shape", [(8 * 3,), (3, 8, 1), (7, 3), (8, 2)])
def test_prefill_lse(shape):
    import paged_kv_flashattention_gb300 as pa
    q = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    pt, cu, g = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.ones(2)
    with pytest.raises(ValueError, match="lse must be"):
        pa.prefill(q, *pools(True), pt, cu, cu, 3, 64, lse=torch.zeros(shape), scheduler=torch.zeros(2, dtype=torch.int32),
                   k_scale=g, v_scale=g, kv_dtype=pa.PA_KV_FP4)
