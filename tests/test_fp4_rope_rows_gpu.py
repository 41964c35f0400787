"""The fused 4-bit rotary store at the full rotated width, and the K rows and
rotated q of a planned batch against a rotation done on the host."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_harness import dev_np
from oracle import fp4
from pa_harness import bf16_dev, bf16_host

pytestmark = pytest.mark.gpu


def rotate(bits, pos, cs, rot, interleaved):
    """include/pa.h's rotation: each product and the sum rounded in fp32, the
    result to bf16; elements past rot copied.  bits uint16 [T, H, d]."""
    x = W.bf16_bits_to_f32(bits).astype(np.float32)
    h = rot // 2
    c, s = cs[pos, None, :h], cs[pos, None, h:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :h], x[..., h:rot])
    u = W.f32_to_bf16_bits((a * c).astype(np.float32) - (b * s).astype(np.float32))
    w = W.f32_to_bf16_bits((b * c).astype(np.float32) + (a * s).astype(np.float32))
    out = bits.copy()
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = u, w
    else:
        out[..., :h], out[..., h:rot] = u, w
    return out


@pytest.mark.parametrize("hq,hkv,d,rot", [(32, 8, 128, 128), (12, 6, 128, 128), (3, 3, 128, 112), (4, 1, 128, 80),
                                          (32, 8, 64, 64), (5, 5, 64, 48), (16, 16, 128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 77])
def test_rows_and_q(cuda_device, hq, hkv, d, rot, interleaved, T):
    """Every byte of both pools and of q, in place and out of place."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(hq + d + rot + T)
    slots, far = 128, 5000
    q, k, v = (W.normal_bf16(rng, (T, h, d)) for h in (hq, hkv, hkv))
    pos = rng.integers(0, far, T).astype(np.int32)
    sm = rng.permutation(slots)[:T].astype(np.int32)
    sm[3::9] = -1
    cs = pa.rope_cos_sin_table(far, rot, 10000.0)
    ks, vs = rng.uniform(1e-3, 3e-3, hkv).astype(np.float32), rng.uniform(1e-3, 3e-3, hkv).astype(np.float32)
    rb = fp4.layout(hkv, d)[-1]
    rows = [rng.integers(0, 256, (slots, rb), dtype=np.uint8) for _ in range(2)]
    pools = [dev_np(r, cuda_device) for r in rows]
    qd = bf16_dev(q, cuda_device)
    for q_out in (torch.zeros_like(qd), qd):
        got = pa.rope_store_kv(qd, bf16_dev(k, cuda_device), bf16_dev(v, cuda_device), dev_np(pos, cuda_device),
                               cs.to(cuda_device), dev_np(sm, cuda_device), *pools, q_out=q_out, interleaved=interleaved,
                               k_scale=dev_np(ks, cuda_device), v_scale=dev_np(vs, cuda_device), kv_dtype=pa.PA_KV_FP4)
        assert np.array_equal(bf16_host(got), rotate(q, pos, cs.numpy(), rot, interleaved))
    fp4.store(W.bf16_bits_to_f32(rotate(k, pos, cs.numpy(), rot, interleaved)), sm, rows[0], ks)
    fp4.store(W.bf16_bits_to_f32(v), sm, rows[1], vs)
    for got, want, what in zip(pools, rows, "KV"):
        bad = np.argwhere(got.cpu().numpy() != want)
        assert bad.size == 0, f"{what} rows: {len(bad)} bytes differ, first at {bad[0]}"
    assert pa.device_error() == 0


@pytest.mark.parametrize("page,hq,hkv,d", [(16, 32, 8, 128), (1, 8, 2, 64)])
def test_planned_prompt(cuda_device, page, hq, hkv, d):
    """Plan, then rotary store: the planned positions rotate q and k, the
    planned slots receive the rows, padded tokens leave nothing."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(98)
    cached, extend = np.array([0, 33, 16, 5], np.int32), np.array([40, 1, 70, 0], np.int32)
    max_k, pad, T = 100, 6, int(extend.sum())
    pages = 4 * (max_k // page + 1)
    order = rng.permutation(pages).astype(np.int32)
    tt = np.full((4, max_k), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(cached):
        j = np.arange(n)
        tt[b, :n] = order[at + j // page] * page + j % page
        at += -(-int(n) // page)
    plan = pa.BatchPlanner(cuda_device, 4, T + pad, max_k, page)
    b = plan.build(dev_np(cached, cuda_device), dev_np(extend, cuda_device), dev_np(tt, cuda_device),
                   torch.arange(4, dtype=torch.int32, device=cuda_device), free_pages=dev_np(order[at:], cuda_device))
    q, k, v = (W.normal_bf16(rng, (T + pad, h, d)) for h in (hq, hkv, hkv))
    cs = pa.rope_cos_sin_table(max_k, d)
    g = np.linspace(1.5e-3, 2.5e-3, hkv).astype(np.float32)
    rb = pa.fp4_row_bytes(hkv, d)
    pools = [torch.full((pages, page, rb), 255, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    got = pa.rope_store_kv(bf16_dev(q, cuda_device), bf16_dev(k, cuda_device), bf16_dev(v, cuda_device), b.positions,
                           cs.to(cuda_device), b.slot_mapping, *pools, k_scale=dev_np(g, cuda_device),
                           v_scale=dev_np(g, cuda_device), kv_dtype=pa.PA_KV_FP4)
    pos = np.concatenate([np.arange(c, c + e) for c, e in zip(cached, extend)] + [np.zeros(pad, int)])
    sm = b.slot_mapping.cpu().numpy()
    assert np.array_equal(bf16_host(got), rotate(q, pos, cs.numpy(), d, False))
    for pool, x in zip(pools, (rotate(k, pos, cs.numpy(), d, False), v)):
        want = np.full((pages * page, rb), 255, np.uint8)
        fp4.store(W.bf16_bits_to_f32(x), sm, want, g)
        assert np.array_equal(pool.view(-1, rb).cpu().numpy(), want)
    assert pa.device_error() == 0
