"""The order in which 4-bit prefill hands out its items (by tile number, or by
class of key positions) changes no bit: the same requests under an exact and
under loose bounds on the keys, with more items than CTAs and with fewer, and
with rows of padding behind the last request."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_harness import FP4Problem, check

pytestmark = pytest.mark.gpu

CASES = {
    "few items": ([0, 300, 20], [130, 1, 40], 4, 2),
    "as many items as CTAs": ([0] * 19, [100] * 19, 16, 4),          # 19 * 8 = 152
    "one more": ([0] * 18 + [500], [100] * 18 + [129], 16, 4),
    "more items": ([0, 3000, 10, 700], [640, 300, 257, 513], 32, 8),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("page", [1, 16])
def test_bounds_and_caps(cuda_device, name, page):
    cached, ext, hq, hkv = CASES[name]
    p = W.small_problem(len(cached) + page, cached, ext, num_q_heads=hq, num_kv_heads=hkv, head_dim=64, page_size=page)
    f = FP4Problem(p, cuda_device, 5)
    m, ref = f.meta, f.oracle()
    first, _ = f.prefill()
    table, exact = m.page_table, m.max_seqlen_k
    for bound in (exact, exact + 128, 20000, 70000):
        wide = torch.full((len(cached), -(-bound // page)), 1 << 30, dtype=torch.int32, device=cuda_device)
        wide[:, :table.shape[1]] = table
        m.page_table, m.max_seqlen_k = wide, bound
        for ctas in (0, 1, 5):
            out, lse = f.prefill(max_ctas=ctas)
            assert torch.equal(out, first), f"{name} P{page} bound {bound} ctas {ctas}"
            check(out, lse, ref, f"{name} P{page} bound {bound} ctas {ctas}")


def test_padded_rows(cuda_device):
    """total_q above the requests' rows (a planned batch): the same bits, and
    the rows behind the last request as they were."""
    import paged_kv_flashattention_gb300 as pa
    cached, ext, hq, hkv = CASES["more items"]
    p = W.small_problem(9, cached, ext, num_q_heads=hq, num_kv_heads=hkv, head_dim=64)
    f = FP4Problem(p, cuda_device, 6)
    m = f.meta
    want, _ = f.prefill()
    n = f.q.shape[0]
    q = torch.cat([f.q, torch.full((1000, hq, 64), float("nan"), dtype=torch.bfloat16, device=cuda_device)])
    out = torch.full_like(q, 3.0)
    pa.prefill(q, f.k_cache, f.v_cache, m.page_table, m.cu_seqlens_q, m.cu_seqlens_k, m.max_seqlen_q, m.max_seqlen_k,
               scale=p.scale, out=out, k_scale=f.k_scale, v_scale=f.v_scale, kv_dtype=pa.PA_KV_FP4)
    assert torch.equal(out[:n], want) and bool((out[n:] == 3).all())
