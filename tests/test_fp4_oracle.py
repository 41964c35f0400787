"""Pins of the 4-bit oracle (no GPU): the format against closed forms and a
second rounding rule, and attention over 4-bit pools against the fp64 oracle
over bf16 pools that hold the same values."""
import numpy as np
import pytest

import oracle
import workloads as W
from oracle import fp4


def test_tables():
    assert fp4.E4M3[0x7E] == 448.0 and fp4.E4M3[0x38] == 1.0 and fp4.E4M3[1] == 2.0 ** -9
    for c in range(127):
        assert fp4.E4M3[c] == oracle.e4m3_value(c)
    assert list(fp4.E2M1) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


@pytest.mark.parametrize("hkv,d,want", [(8, 128, 576), (8, 64, 288), (1, 128, 80), (1, 64, 48), (2, 128, 144),
                                        (2, 64, 80), (6, 64, 240), (32, 128, 2304), (12, 128, 864)])
def test_row_bytes(hkv, d, want):
    assert fp4.layout(hkv, d)[-1] == want
    import paged_kv_flashattention_gb300 as pa
    from paged_kv_flashattention_gb300 import build
    build.build()
    assert pa.fp4_row_bytes(hkv, d) == want


def test_row_bytes_refusals():
    import paged_kv_flashattention_gb300 as pa
    for hkv, d in ((8, 96), (0, 64), (8, -64), (64, 128)):
        with pytest.raises(ValueError):
            pa.fp4_row_bytes(hkv, d)


def test_nearest_code_ties_and_ends():
    x = [0.25, 0.2500001, 0.75, 0.7499999, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 6.0, 100.0, np.inf, 0.0]
    assert fp4.nearest_code(np.array(x), fp4.E2M1).tolist() == [0, 1, 2, 1, 2, 4, 4, 6, 6, 7, 7, 7, 7, 0]


def test_scale_codes_match_the_fp8_encoder():
    rng = np.random.default_rng(5)
    x = np.exp(rng.uniform(-9, 8, 4000)).astype(np.float32)
    want = [oracle.e4m3_encode(float(v)) for v in x]
    assert fp4.nearest_code(x, fp4.E4M3).tolist() == want


def test_quantise_is_nearest_and_packs():
    """Every element's error is within half a step of its place on the grid;
    pack and unpack are inverse; blocks of zeros, NaN and infinities."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((50, 6, 64)).astype(np.float32)
    g = rng.uniform(0.002, 0.003, 6).astype(np.float32)
    codes, scales = fp4.quantise(x, g)
    v = fp4.unpack(fp4.pack(codes, scales), 6, 64, g)
    step = np.repeat(fp4.E4M3[scales], 16, -1) * g[None, :, None].astype(np.float64)
    z = np.abs(x) / step
    half = np.where(z <= 2, 0.25, np.where(z <= 4, 0.5, 1.0))
    over = np.maximum(z - 6.0, 0.0)           # a scale rounded down saturates the largest
    assert np.all(np.abs(v - x) <= step * (np.maximum(half, over) + 1e-6))
    assert np.all(z < 6.5)
    x[0, 0, :16] = 0
    x[1, 1, 3] = np.nan
    x[2, 2, 4], x[2, 2, 5] = np.inf, -np.inf
    codes, scales = fp4.quantise(x, g)
    assert scales[0, 0, 0] == 0 and not codes[0, 0, :16].any()
    assert scales[1, 1, 0] == 127 and scales[2, 2, 0] == 0x7E
    assert codes[2, 2, 4] == 7 and codes[2, 2, 5] == 15


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 9), (False, 0)])
def test_attention_equals_the_bf16_oracle(causal, window):
    """code * scale has at most six bits, so a bf16 pool can hold it; with
    head scales of 1 both oracles compute the same attention."""
    p = W.small_problem(77, [5, 0, 40], [3, 17, 30], num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16,
                        causal=causal)
    rng = np.random.default_rng(8)
    hkv, d = 2, 64
    slots = p.num_pages * 16
    one = np.ones(hkv, np.float32)
    rows = [fp4.pack(*fp4.quantise(rng.standard_normal((slots, hkv, d)).astype(np.float32) * 50, one)) for _ in range(2)]
    vals = [fp4.unpack(r, hkv, d, one) for r in rows]
    bits = [W.f32_to_bf16_bits(v.astype(np.float32)) for v in vals]
    for b, v in zip(bits, vals):
        assert np.array_equal(W.bf16_bits_to_f32(b).astype(np.float64), v)
    cu_q, cu_k, _, _, mk = oracle.seqlens(p.cached_len, p.extend_len)[:5]
    pt = oracle.page_table_from_token_table(p.token_table, p.table_idx, mk, 16)
    q = W.bf16_bits_to_f32(p.q)
    o, l, _ = fp4.attention(q, rows[0], rows[1], pt, cu_q, cu_k, num_kv_heads=hkv, page_size=16, k_scale=one, v_scale=one,
                         scale=0.01, causal=causal, window=window)
    shape = (p.num_pages, 16, hkv, d)
    kw = dict(window_left=window - 1) if window else {}
    want, want_l = oracle.attention(p.q, bits[0].reshape(shape), bits[1].reshape(shape), pt, cu_q, cu_k, num_q_heads=8,
                                    num_kv_heads=hkv, head_dim=d, page_size=16, causal=causal, scale=0.01, **kw)
    assert np.abs(o - want.reshape(o.shape)).max() < 1e-11 * 50
    assert np.abs(l - want_l.reshape(l.shape)).max() < 1e-11
