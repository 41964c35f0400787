"""Attention over 4-bit pools with one dominant key over 32768 small weights,
where weights held in f16 lose the most.

A weight is rounded to f16 relative to the running maximum m of its range: by
half a step, 2^-11 of itself in f16's normal range and 2^-25 of exp(m) below
it (f16's subnormal spacing is 2^-24), down to zero.  So beside the bounds of
fp4_harness an output may be off by 2^-25 sum_j |V_j| exp(m - lse), m at most
the row's largest score: 2^-25 * 32768 = 2^-10 of the largest |V| at the
worst.  The head scales of K spread the dominant key 5 to 20 (natural units)
above the rest, across f16's subnormal range (2^-14 = e^-9.7) and its end
(2^-25 = e^-17.3), where every small weight errs to the same side.  The scores:
sum |q k| scale is at most 20, within fp4_harness's 40."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_harness import TOL_A, TOL_LSE, dev_np
from oracle import fp4
from pa_harness import bf16_dev

pytestmark = pytest.mark.gpu

N = 32768
GAPS = np.array([5.0, 9.0, 11.0, 14.0, 16.5, 17.0, 17.5, 20.0])


def case(dev, d, at):
    rng = np.random.default_rng(d + at)
    hkv = len(GAPS)
    codes = np.zeros((N, hkv, d), np.uint8)
    codes[at] = 7                                              # 6 in every element
    scales = np.full((N, hkv, d // 16), 0x38, np.uint8)        # 1
    kr = fp4.pack(codes, scales, np.zeros((N, fp4.layout(hkv, d)[-1]), np.uint8))
    vcodes = rng.integers(1, 8, (N, hkv, d)).astype(np.uint8)  # positive, so that the errors add up
    vcodes[at] = 15                                            # -6
    vr = fp4.pack(vcodes, scales, np.zeros_like(kr))
    ks = (GAPS / (6.0 * d ** 0.5)).astype(np.float32)          # scale * sum of d products 1 * 6 * ks = gap
    vs = np.full(hkv, 0.25, np.float32)
    q = np.full((1, hkv, d), 0x3F80, np.uint16)                # 1.0
    ref = fp4.attention(W.bf16_bits_to_f32(q), kr, vr, np.arange(N // 16)[None], [0, 1], [0, N], num_kv_heads=hkv,
                        page_size=16, k_scale=ks, v_scale=vs, scale=d ** -0.5)
    vmag = np.abs(fp4.unpack(vr, hkv, d, vs)).sum(0)           # [Hkv, d]
    small = 2.0 ** -25 * vmag * np.exp(GAPS - ref[1][0])[:, None]
    args = [dev_np(kr, dev).view(N // 16, 16, -1), dev_np(vr, dev).view(N // 16, 16, -1),
            torch.arange(N // 16, dtype=torch.int32, device=dev)[None].contiguous()]
    return bf16_dev(q, dev), args, dict(scale=d ** -0.5, k_scale=dev_np(ks, dev), v_scale=dev_np(vs, dev)), ref, small


def compare(out, lse, ref, small, what):
    got = out.float().cpu().numpy().astype(np.float64)
    over = np.abs(got - ref[0]) - (2.0 ** -8 * np.abs(ref[0]) + TOL_A * ref[2] + small)
    assert over.max() <= 0, f"{what}: {np.count_nonzero(over > 0)} outputs off, worst by {over.max():.3g} of the bound"
    assert np.abs(lse.cpu().numpy() - ref[1]).max() <= TOL_LSE, what


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 12345, N - 1])
def test_decode(cuda_device, d, at):
    import paged_kv_flashattention_gb300 as pa
    q, args, kw, ref, small = case(cuda_device, d, at)
    lens = torch.tensor([N], dtype=torch.int32, device=cuda_device)
    for chunk in (0, N):                                       # many ranges; one
        lse = torch.empty((1, len(GAPS)), device=cuda_device)
        out = pa.decode(q, *args, lens, N, lse=lse, kv_chunk=chunk, kv_dtype=pa.PA_KV_FP4, **kw)
        compare(out, lse, ref, small, f"decode d{d} at {at} chunk {chunk}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 12345, N - 1])
def test_prefill(cuda_device, d, at):
    import paged_kv_flashattention_gb300 as pa
    q, args, kw, ref, small = case(cuda_device, d, at)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=cuda_device) for n in (1, N))
    lse = torch.empty((len(GAPS), 1), device=cuda_device)
    out = pa.prefill(q, *args, cu_q, cu_k, 1, N, lse=lse, kv_dtype=pa.PA_KV_FP4, **kw)
    compare(out, lse.t(), ref, small, f"prefill d{d} at {at}")
