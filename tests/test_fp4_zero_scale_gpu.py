"""Attention over 4-bit pools whose K or V head scales are zero (an all-zero
head's largest magnitude / 2688) or lie below fp32's normal range: every key of
such a head scores zero, so its rows are the plain mean of the visible values."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_harness import FP4Problem, check, dev_np

pytestmark = pytest.mark.gpu


def rescale(f, ks, vs):
    f.ks, f.vs = f.ks.copy(), f.vs.copy()
    for at, x in ks.items():
        f.ks[at] = x
    for at, x in vs.items():
        f.vs[at] = x
    f.k_scale, f.v_scale = dev_np(f.ks, f.dev), dev_np(f.vs, f.dev)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [0, 21])
def test_decode(cuda_device, d, page, window):
    import paged_kv_flashattention_gb300 as pa
    L = np.array([1, 7, 16, 17, 40, 333, 700], np.int32)
    p = W.small_problem(81 + d, L - 1, np.ones_like(L), num_q_heads=32, num_kv_heads=8, head_dim=d, page_size=page)
    f = FP4Problem(p, cuda_device, 82)
    rescale(f, {0: 0.0, 3: 1e-40, 7: 1e-38}, {1: 0.0})
    out, lse = f.decode(sliding_window=window)
    check(out, lse, f.oracle(window=window), f"zero scales d{d} P{page} window {window}")
    assert pa.device_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 8, 64)])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [0, 21])
def test_prefill(cuda_device, hq, hkv, d, page, window):
    import paged_kv_flashattention_gb300 as pa
    p = W.small_problem(83 + d, [0, 5, 130, 300], [40, 1, 129, 77], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                        page_size=page)
    f = FP4Problem(p, cuda_device, 84)
    rescale(f, {0: 0.0}, {1: 0.0})
    out, lse = f.prefill(sliding_window=window)
    check(out, lse, f.oracle(window=window), f"zero scales {hq}/{hkv} d{d} P{page} window {window}")
    assert pa.device_error() == 0


@pytest.mark.parametrize("kernel", ["decode", "prefill"])
def test_nan_scale_stays_nan(cuda_device, kernel):
    """A NaN head scale is not mistaken for a tiny one."""
    L = np.array([40, 100], np.int32)
    p = W.small_problem(85, L - 1, np.ones_like(L), num_q_heads=8, num_kv_heads=4, head_dim=128)
    f = FP4Problem(p, cuda_device, 86)
    rescale(f, {2: np.nan}, {})
    out, _ = getattr(f, kernel)()
    want = torch.zeros_like(out, dtype=torch.bool)
    want[:, 4:6] = True
    assert torch.equal(torch.isnan(out), want)


def test_store(cuda_device):
    """A head of zero scale stores codes of zero, whatever its values, and reads
    back as zeros; the heads beside it keep theirs."""
    import paged_kv_flashattention_gb300 as pa
    hkv, d, T = 4, 64, 9
    x = torch.randn((T, hkv, d), device=cuda_device).bfloat16()
    x[:, 1] = 0                                                # all zeros at scale zero, and head 2 not
    g = torch.tensor([2e-3, 0.0, 0.0, 2e-3], device=cuda_device)
    pools = [torch.full((16, pa.fp4_row_bytes(hkv, d)), 255, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int32, device=cuda_device)
    pa.store_kv_fp4(x, x, slots, *pools, g, g)
    for back in pa.load_kv_fp4(slots, *pools, g, g, d):
        assert not back[:, 1:3].any()
        assert bool(torch.isfinite(back).all()) and bool((back[:, [0, 3]].float().abs().amax(-1) > 0.5).all())
