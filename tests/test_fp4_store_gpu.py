"""GPU parity of the 4-bit store, the rotary fused with it and the read-back
against the oracle: pool bytes are equal bit for bit (the format fixes every
rounding), and a row read back is the exact value rounded as documented."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from oracle import fp4
from pa_harness import bf16_dev, bf16_host

pytestmark = pytest.mark.gpu


def dev_u8(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def wide_bf16(rng, shape):
    """bf16 bits over many binades, with zeros, subnormals and exact ties."""
    x = W.normal_bf16(rng, shape).reshape(-1)
    pick = rng.integers(0, 8, x.size)
    expo = rng.integers(100, 150, x.size).astype(np.uint16) << 7
    x = np.where(pick == 0, (x & 0x807F) | expo, x)
    x = np.where(pick == 1, x & 0x8000, x)
    x = np.where(pick == 2, x & 0xFF80, x)               # powers of two: ties after a power-of-two step
    return x.astype(np.uint16).reshape(shape)


def same(got, want, what):
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{what}: {len(bad)} of {want.size} bytes differ, first at {bad[0]}: " \
                          f"{got[tuple(bad[0])]:#x}, expected {want[tuple(bad[0])]:#x}"


def expect_rows(bits, slots, pool, scale):
    fp4.store(W.bf16_bits_to_f32(bits), slots, pool, scale)


@pytest.mark.parametrize("hkv,d", [(8, 128), (8, 64), (1, 128), (1, 64), (2, 64), (6, 64), (12, 128), (16, 64), (32, 128)])
@pytest.mark.parametrize("T", [0, 1, 7, 300])
def test_store_and_load(cuda_device, hkv, d, T):
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(1000 * hkv + d + T)
    k, v = wide_bf16(rng, (T, hkv, d)), wide_bf16(rng, (T, hkv, d))
    if T > 3:
        k[1, 0, 5] = 0x7FC0                              # NaN
        v[2, 0, :3] = [0x7F80, 0xFF80, 0x3F80]           # infinities
        v[3] = 0
    slots = 512
    ks = np.exp2(rng.integers(-12, -6, hkv)).astype(np.float32)      # exact steps: ties happen
    vs = rng.uniform(1e-3, 3e-3, hkv).astype(np.float32)
    sm = rng.permutation(slots)[:T].astype(np.int32)
    sm[::5] = -1
    rb = fp4.layout(hkv, d)[-1]
    kc, vc = rng.integers(0, 256, (slots, rb), dtype=np.uint8), rng.integers(0, 256, (slots, rb), dtype=np.uint8)
    kd, vd = dev_u8(kc, cuda_device).view(slots // 16, 16, rb), dev_u8(vc, cuda_device).view(slots // 16, 16, rb)
    ksd, vsd, smd = dev_u8(ks, cuda_device), dev_u8(vs, cuda_device), dev_u8(sm, cuda_device)
    pa.store_kv_fp4(bf16_dev(k, cuda_device), bf16_dev(v, cuda_device), smd, kd, vd, ksd, vsd)
    expect_rows(k, sm, kc, ks)
    expect_rows(v, sm, vc, vs)
    same(kd.cpu().numpy().reshape(slots, rb), kc, "K rows")
    same(vd.cpu().numpy().reshape(slots, rb), vc, "V rows")
    assert pa.device_error() == 0
    # every slot twice over and the skipped ones: one fp32 product and one bf16 rounding
    if T:
        at = np.concatenate([sm, sm[::-1]])
        ko, vo = pa.load_kv_fp4(dev_u8(at, cuda_device), kd, vd, ksd, vsd, d)
        for got, pool, g in ((ko, kc, ks), (vo, vc, vs)):
            one = np.ones(hkv, np.float32)
            with np.errstate(all="ignore"):
                exact = fp4.unpack(pool[np.maximum(at, 0)], hkv, d, one).astype(np.float32) * g[None, :, None]
            want = np.where((at >= 0)[:, None, None], exact, np.float32(0)).astype(np.float32)
            gotf = W.bf16_bits_to_f32(bf16_host(got))
            ref = W.bf16_bits_to_f32(W.f32_to_bf16_bits(np.nan_to_num(want, nan=0.0)))
            ref = np.where(np.isnan(want), np.nan, ref)
            assert np.array_equal(gotf, ref, equal_nan=True)


def test_border_step(cuda_device):
    """Steps whose significand is all ones, and their neighbours, against
    elements at every border of the codes: the quotient that decides is the
    IEEE one."""
    import paged_kv_flashattention_gb300 as pa
    hkv, d = 8, 64
    ones = np.array([0x3F7FFFFF, 0x3F7FFFFE, 0x3F800000, 0x3F800001, 0x3FBFFFFF, 0x3FC00000, 0x3FC00001, 0x3F000000],
                    np.uint32).view(np.float32)
    T = 64
    x = np.zeros((T, hkv, d), np.float32)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0])
    for t in range(T):
        x[t] = np.tile(borders, d // 16) * 2.0 ** (t - 32)
    bits = W.f32_to_bf16_bits(x.astype(np.float32))
    g = (ones * np.float32(2.0 ** -7)).astype(np.float32)
    sm = np.arange(T, dtype=np.int32)
    rb = fp4.layout(hkv, d)[-1]
    pool = np.zeros((T, rb), np.uint8)
    kd, vd = dev_u8(pool, cuda_device), dev_u8(pool, cuda_device)
    pa.store_kv_fp4(bf16_dev(bits, cuda_device), bf16_dev(bits, cuda_device), dev_u8(sm, cuda_device), kd, vd,
                    dev_u8(g, cuda_device), dev_u8(g, cuda_device))
    expect_rows(bits, sm, pool, g)
    same(kd.cpu().numpy(), pool, "K rows")
    same(vd.cpu().numpy(), pool, "V rows")


@pytest.mark.parametrize("g", [1e-38, 3e-42, 1e36, 3e38])
def test_extreme_head_scales(cuda_device, g):
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(3)
    hkv, d, T = 2, 64, 40
    bits = wide_bf16(rng, (T, hkv, d))
    bits[::2] = (bits[::2] & 0x807F) | (rng.integers(1, 254, bits[::2].shape).astype(np.uint16) << 7)
    gs = np.full(hkv, g, np.float32)
    sm = np.arange(T, dtype=np.int32)
    rb = fp4.layout(hkv, d)[-1]
    pool = np.zeros((T, rb), np.uint8)
    kd, vd = dev_u8(pool, cuda_device), dev_u8(pool, cuda_device)
    gd = dev_u8(gs, cuda_device)
    pa.store_kv_fp4(bf16_dev(bits, cuda_device), bf16_dev(bits, cuda_device), dev_u8(sm, cuda_device), kd, vd, gd, gd)
    expect_rows(bits, sm, pool, gs)
    same(kd.cpu().numpy(), pool, "K rows")


def test_slots_outside_the_pool(cuda_device):
    """A slot past the pool is not written and raises the error bit; reading it
    gives zeros."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(4)
    hkv, d, slots = 4, 128, 64
    k = bf16_dev(W.normal_bf16(rng, (3, hkv, d)), cuda_device)
    rb = pa.fp4_row_bytes(hkv, d)
    pool = torch.zeros((slots, rb), dtype=torch.uint8, device=cuda_device)
    g = torch.full((hkv,), 2e-3, device=cuda_device)
    sm = torch.tensor([3, slots, -1], dtype=torch.int32, device=cuda_device)
    pa.store_kv_fp4(k, k, sm, pool, pool.clone(), g, g)
    assert pa.device_error() == pa.PA_DEVERR_PAGE_RANGE
    assert pool[3].any() and not pool[:3].any() and not pool[4:].any()
    a, _ = pa.load_kv_fp4(sm, pool, pool, g, g, d)
    assert pa.device_error() == pa.PA_DEVERR_PAGE_RANGE
    assert a[0].any() and not a[1:].any()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 1, 64), (12, 6, 64), (16, 16, 128)])
@pytest.mark.parametrize("rot", [16, 32, 48, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_store_equals_the_chain(cuda_device, hq, hkv, d, rot, interleaved):
    """The fused call equals the bf16 rotary store followed by the 4-bit
    store of the rotated keys, bit for bit, in place and out of place, with
    skipped slots and a position outside the table."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(hq + d + rot)
    T, slots, far = 77, 128, 900
    q = bf16_dev(W.normal_bf16(rng, (T, hq, d)), cuda_device)
    k = bf16_dev(W.normal_bf16(rng, (T, hkv, d)), cuda_device)
    v = bf16_dev(W.normal_bf16(rng, (T, hkv, d)), cuda_device)
    pos = rng.integers(0, far, T).astype(np.int32)
    pos[5] = far
    sm = rng.permutation(slots)[:T].astype(np.int32)
    sm[::9] = -1
    cs = pa.rope_cos_sin_table(far, rot, 10000.0).to(cuda_device)
    posd, smd = dev_u8(pos, cuda_device), dev_u8(sm, cuda_device)
    g = torch.full((hkv,), 2e-3, device=cuda_device)
    rb = pa.fp4_row_bytes(hkv, d)
    pools = [torch.zeros((slots, rb), dtype=torch.uint8, device=cuda_device) for _ in range(4)]
    # the chain: rotate into a bf16 pool at slot t, then quantise
    k16 = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device=cuda_device)
    v16 = torch.zeros_like(k16)
    iota = torch.arange(T, dtype=torch.int32, device=cuda_device)
    want_q = pa.rope_store_kv(q, k, v, posd, cs, iota, k16, v16, interleaved=interleaved, q_out=q.clone())
    sm2 = sm.copy()
    sm2[5] = -1
    pa.store_kv_fp4(k16, v, dev_u8(sm2, cuda_device), pools[0], pools[1], g, g)
    assert pa.device_error() == pa.PA_DEVERR_POSITION
    got = pa.rope_store_kv(q, k, v, posd, cs, smd, pools[2], pools[3], interleaved=interleaved, q_out=q.clone(),
                           k_scale=g, v_scale=g, kv_dtype=pa.PA_KV_FP4)
    assert pa.device_error() == pa.PA_DEVERR_POSITION
    assert torch.equal(got.view(torch.int16), want_q.view(torch.int16))
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    qi = q.clone()
    pa.rope_store_kv(qi, k, v, posd, cs, smd, pools[2], pools[3], interleaved=interleaved, q_out=qi, k_scale=g,
                     v_scale=g, kv_dtype=pa.PA_KV_FP4)
    pa.device_error()
    assert torch.equal(qi.view(torch.int16), want_q.view(torch.int16))


def test_store_in_a_graph_and_on_a_stream(cuda_device):
    """Captured and replayed with new values in the same buffers."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(9)
    hkv, d, T = 8, 128, 33
    k = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device=cuda_device)
    sm = torch.arange(T, dtype=torch.int32, device=cuda_device)
    pool = torch.zeros((64, pa.fp4_row_bytes(hkv, d)), dtype=torch.uint8, device=cuda_device)
    pool2, g = pool.clone(), torch.full((hkv,), 2e-3, device=cuda_device)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pa.store_kv_fp4(k, k, sm, pool, pool2, g, g)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pa.store_kv_fp4(k, k, sm, pool, pool2, g, g)
    for n in range(2):
        bits = W.normal_bf16(rng, (T, hkv, d))
        k.copy_(bf16_dev(bits, cuda_device))
        graph.replay()
        torch.cuda.synchronize()
        want = np.zeros(tuple(pool.shape), np.uint8)
        expect_rows(bits, np.arange(T), want, g.cpu().numpy())
        assert np.array_equal(pool.cpu().numpy(), want) and np.array_equal(pool2.cpu().numpy(), want)
