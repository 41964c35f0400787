"""Refusals of the 4-bit entry points and of the batch plan, on the host: the
C calls run in a child process that sees no GPU (their pointers are made up),
the binding's checks on CPU tensors."""
import json
import os
import subprocess
import sys

import pytest
import torch

import fp4_reject_cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rejections():
    from paged_kv_flashattention_gb300 import build
    build.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "fp4_reject_cases.py")],
                       capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("case", sorted(fp4_reject_cases.expected()))
def test_rejects_before_launch(rejections, case):
    status, message = rejections[case]
    want = fp4_reject_cases.expected()[case]
    assert status == want, f"{case}: status {status} ({message}), expected {want}"
    if want != 0:
        assert message, f"{case}: no error message"


def _pools(hkv=8, d=64, pages=4, page=16):
    import paged_kv_flashattention_gb300 as pa
    return [torch.zeros((pages, page, pa.fp4_row_bytes(hkv, d)), dtype=torch.uint8) for _ in range(2)]


def test_binding_store_checks():
    import paged_kv_flashattention_gb300 as pa
    kc, vc = _pools()
    k = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    sm = torch.zeros(3, dtype=torch.int32)
    g = torch.ones(8)
    with pytest.raises(TypeError):
        pa.store_kv_fp4(k.float(), k, sm, kc, vc, g, g)
    with pytest.raises(TypeError):
        pa.store_kv_fp4(k, k, sm, kc.view(torch.int8), vc, g, g)
    with pytest.raises(ValueError):
        pa.store_kv_fp4(k, k, sm[:2], kc, vc, g, g)
    with pytest.raises(ValueError):
        pa.store_kv_fp4(k, k, sm, kc, vc, g[:7], g)
    with pytest.raises(ValueError):
        pa.store_kv_fp4(k, k, sm, kc[..., :-16].contiguous(), vc[..., :-16].contiguous(), g, g)
    with pytest.raises(ValueError):
        pa.store_kv_fp4(k, k, sm, kc, vc[:2], g, g)
    with pytest.raises(ValueError):
        pa.store_kv_fp4(k.transpose(0, 1).contiguous().transpose(0, 1), k, sm, kc, vc, g, g)
    with pytest.raises(ValueError):
        pa.load_kv_fp4(sm, kc, vc, g, g, 128)
    with pytest.raises(ValueError):
        pa.load_kv_fp4(sm, kc, vc, g, g, 64, k_out=k[:2])
    with pytest.raises(ValueError):
        pa.load_kv_fp4(sm, kc, vc, None, g, 64)


def test_binding_kv_dtype_checks():
    """4-bit rows are used only where the caller says so, and a kv_dtype that
    the pools are not is refused."""
    from paged_kv_flashattention_gb300 import api
    u8, b16 = torch.zeros(4, dtype=torch.uint8), torch.zeros(4, dtype=torch.bfloat16)
    assert api._kv_dtype(u8, u8) == api.PA_KV_FP8_E4M3
    assert api._kv_dtype(u8, u8, api.PA_KV_FP4) == api.PA_KV_FP4
    assert api._kv_dtype(b16, b16, api.PA_KV_BF16) == api.PA_KV_BF16
    for pool, asked in ((b16, api.PA_KV_FP4), (u8, api.PA_KV_BF16), (b16, api.PA_KV_FP8_E4M3)):
        with pytest.raises(TypeError):
            api._kv_dtype(pool, pool, asked)
    with pytest.raises(ValueError):
        api._kv_dtype(u8, u8, 3)


def test_binding_batch_checks():
    import paged_kv_flashattention_gb300 as pa
    pl = pa.BatchPlanner("cpu", 4, 16, 100, 16)
    assert pl.page_table.shape == (4, 7) and bool((pl.page_table == -1).all())
    c = torch.zeros(3, dtype=torch.int32)
    tt, idx = torch.zeros((5, 100), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        pl.build(torch.zeros(5, dtype=torch.int32), c, tt, idx)           # more than the planner holds
    with pytest.raises(ValueError):
        pl.build(c, c[:2], tt, idx)
    with pytest.raises(ValueError):
        pl.build(c, c, tt[:, :99], idx)                                   # narrower than max_seqlen_k
    with pytest.raises(TypeError):
        pl.build(c.long(), c, tt, idx)
    with pytest.raises(TypeError):
        pl.build(c, c, tt, idx, free_pages=torch.zeros(4))
    with pytest.raises(ValueError):
        pl.build(c, c, tt.t().contiguous().t(), idx)
    with pytest.raises(ValueError):
        pl.build(c, c, tt[:1].expand(5, 100), idx)                        # rows on top of each other
    for bad in ((-1, 1, 1, 1), (1, 1, 1, 0)):
        with pytest.raises(ValueError):
            pa.BatchPlanner("cpu", *bad)


def test_binding_decode_sizes():
    import paged_kv_flashattention_gb300 as pa
    kc, _ = _pools(pages=300)
    shape = (3, 32, 64)
    n = pa.decode_workspace_size(shape, kc, 4096, kv_dtype=pa.PA_KV_FP4, num_kv_heads=8)
    assert n > 0 and pa.decode_kv_chunk(shape, kc, 4096, kv_dtype=pa.PA_KV_FP4, num_kv_heads=8) % 16 == 0
    flat = kc.view(-1, kc.shape[-1])
    assert n == pa.decode_workspace_size(shape, flat, 4096, page_size=16, kv_dtype=pa.PA_KV_FP4, num_kv_heads=8)
    with pytest.raises(ValueError):
        pa.decode_workspace_size(shape, kc, 4096, kv_dtype=pa.PA_KV_FP4)
    with pytest.raises(ValueError):
        pa.decode_workspace_size(shape, flat, 4096, kv_dtype=pa.PA_KV_FP4, num_kv_heads=8)


def test_binding_attention_checks():
    """Arrays that are too small for the call are refused before any launch."""
    import paged_kv_flashattention_gb300 as pa
    kc, vc = _pools(hkv=2, d=64)
    g = torch.ones(2)
    q = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    pt, lens, cu = (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (3,), (4,)))
    sched = torch.zeros(2, dtype=torch.int32)
    kw = dict(k_scale=g, v_scale=g, kv_dtype=pa.PA_KV_FP4)

    def refused(fn, *a, error=ValueError, **over):
        with pytest.raises(error):
            fn(*a, **{**kw, **over})

    for fn in (pa.decode, pa.decode_noalloc):
        refused(fn, q, kc, vc, pt[:2], lens, 64)
        refused(fn, q, kc, vc, pt, lens[:2], 64)
        refused(fn, q, kc, vc, pt, lens, 64, out=q[:2])
        refused(fn, q, kc, vc, pt, lens, 64, lse=torch.zeros((2, 8)))
        refused(fn, q, kc, vc, pt, lens, 64, k_scale=None)
        refused(fn, q, kc, vc, pt, lens, 64, k_scale=g[:1], v_scale=g[:1])    # rows of another length
        refused(fn, q, kc, vc, pt, lens, 64, page_size=1)
        refused(fn, q[..., :32].contiguous(), kc, vc, pt, lens, 64)
        refused(fn, q, kc.view(torch.int8), vc, pt, lens, 64, error=TypeError)
    pre = (q, kc, vc, pt, cu, cu, 3, 64)
    refused(pa.prefill, *pre[:3], pt[:2], *pre[4:], scheduler=sched)
    refused(pa.prefill, *pre[:5], cu[:3], *pre[6:], scheduler=sched)
    refused(pa.prefill, *pre, scheduler=sched, out=q[:2])
    refused(pa.prefill, *pre, scheduler=sched, lse=torch.zeros((8, 2)))
    refused(pa.prefill, *pre, scheduler=sched, v_scale=g[:1])
    refused(pa.prefill, *pre, scheduler=sched[:1])
    refused(pa.DecodeGraphRunner, kc, vc, num_q_heads=8, max_seqlen_k=64)                         # no head_dim
    refused(pa.DecodeGraphRunner, kc, vc, num_q_heads=8, max_seqlen_k=64, head_dim=64, v_scale=None)
    refused(pa.DecodeGraphRunner, kc, vc, num_q_heads=8, max_seqlen_k=64, head_dim=128)
