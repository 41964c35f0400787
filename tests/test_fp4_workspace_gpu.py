"""One workspace for batches of any size up to its own, on the device: the
host checks with this GPU's SM count, the graph runner with buckets that are no
powers of two, and one buffer used by ever smaller batches."""
import numpy as np
import pytest
import torch

import fp4_workspace as F
import workloads as W
from fp4_harness import FP4Problem, check

pytestmark = pytest.mark.gpu


def test_reported_sizes(cuda_device):
    """(The refused calls launch nothing.)"""
    F.check_smaller_batches()
    F.check_shorter_bounds_and_windows()
    F.check_not_wasteful()
    F.check_given_ranges()


def problem(dev, d, seed, B, hi):
    rng = np.random.default_rng(seed)
    L = rng.integers(1, hi, B).astype(np.int32)
    p = W.small_problem(seed, L - 1, np.ones_like(L), num_q_heads=32, num_kv_heads=8, head_dim=d)
    return FP4Problem(p, dev, seed + 1), L


def wide_table(f, keys):
    """The page table widened to a bound of `keys`."""
    pt = torch.zeros((f.meta.page_table.shape[0], keys // 16), dtype=torch.int32, device=f.dev)
    pt[:, :f.meta.page_table.shape[1]] = f.meta.page_table
    return pt


@pytest.mark.parametrize("keys", [4096, 6080, 8192])
def test_runner_buckets(cuda_device, keys):
    import paged_kv_flashattention_gb300 as pa
    f, L = problem(cuda_device, 128, keys, 5, 900)
    ref, pt = f.oracle(), wide_table(f, keys)
    runner = pa.DecodeGraphRunner(f.k_cache, f.v_cache, num_q_heads=32, max_seqlen_k=keys, buckets=(1, 2, 3, 4, 5),
                                  scale=f.p.scale, k_scale=f.k_scale, v_scale=f.v_scale, kv_dtype=pa.PA_KV_FP4, head_dim=128)
    runner.capture()
    for B in (5, 4, 3, 2, 1):
        out, lse = runner.run(L[:B], q=f.q[:B], page_table=pt[:B])
        torch.cuda.synchronize()
        check(out, lse, tuple(x[:B] for x in ref), f"bucket {B} of {keys} keys")
    assert pa.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 100])
def test_one_buffer_for_smaller_batches(cuda_device, d, window):
    """The bytes behind the reported size stay as they were."""
    import paged_kv_flashattention_gb300 as pa
    keys, B = 4096, 32
    f, L = problem(cuda_device, d, 71, B, 300)
    ref, pt = f.oracle(window=window), wide_table(f, keys)
    need = pa.decode_workspace_size((B, 32, d), f.k_cache, keys, kv_dtype=pa.PA_KV_FP4, num_kv_heads=8)
    buf = torch.full((need + 4096,), 171, dtype=torch.uint8, device=cuda_device)
    lse = torch.empty((B, 32), device=cuda_device)
    for n in (32, 31, 17, 8, 5, 4, 3, 2, 1):
        out = pa.decode(f.q[:n], f.k_cache, f.v_cache, pt[:n], f.meta.cache_seqlens[:n], keys, scale=f.p.scale, lse=lse[:n],
                        workspace=buf[:need], sliding_window=window, k_scale=f.k_scale, v_scale=f.v_scale,
                        kv_dtype=pa.PA_KV_FP4)
        check(out, lse[:n], tuple(x[:n] for x in ref), f"{n} sequences, window {window}")
    assert bool((buf[need:] == 171).all())
    assert pa.device_error() == 0
