"""GPU parity of decode over 4-bit pools against the fp64 oracle (tolerances:
fp4_harness), and the calls around it: windows, long contexts, pools past 32
bits, bad pages, graphs, determinism."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_harness import FP4Problem, check, dev_np, random_rows
from oracle import fp4

pytestmark = pytest.mark.gpu

LENS = [1, 15, 16, 17, 33, 100, 257, 640]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (16, 4), (12, 6), (8, 1), (3, 3), (64, 16), (24, 12)])
@pytest.mark.parametrize("page", [1, 16])
def test_edge_matrix(cuda_device, d, hq, hkv, page):
    import paged_kv_flashattention_gb300 as pa
    L = np.array(LENS, np.int32)
    f = FP4Problem(W.small_problem(100 + d + hq + page, L - 1, np.ones_like(L), num_q_heads=hq, num_kv_heads=hkv,
                                   head_dim=d, page_size=page), cuda_device, hq + d)
    ref = f.oracle()
    for chunk in (0, 16, 48):
        out, lse = f.decode(kv_chunk=chunk)
        check(out, lse, ref, f"d{d} {hq}/{hkv} P{page} chunk {chunk}")
    assert pa.device_error() == 0


def test_empty_rows_and_one_key(cuda_device):
    """Sequences without a key between others: zeros and -inf."""
    p = W.small_problem(7, [0, 40, 0, 7, 0], [1, 1, 1, 1, 1], num_q_heads=32, num_kv_heads=8, head_dim=128)
    f = FP4Problem(p, cuda_device, 8)
    lens = np.array([1, 41, 0, 8, 0], np.int32)
    f.meta.cache_seqlens = dev_np(lens, cuda_device)
    out, lse = f.decode()
    want, want_l, mag = f.oracle()
    for b in (2, 4):
        want[b], want_l[b], mag[b] = 0, -np.inf, 0
    check(out, lse, (want, want_l, mag), "empty rows")


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 5000])
def test_windows(cuda_device, page, window):
    """Only the last keys are read: the table entries of pages before the
    window point outside the pool."""
    import paged_kv_flashattention_gb300 as pa
    L = np.array([1, 16, 31, 100, 333, 1000], np.int32)
    p = W.small_problem(40 + window, L - 1, np.ones_like(L), num_q_heads=16, num_kv_heads=8, head_dim=128, page_size=page)
    f = FP4Problem(p, cuda_device, window)
    ref = f.oracle(window=window)
    pt = f.meta.page_table.clone()
    for b, n in enumerate(L):
        pt[b, :max(0, int(n) - window) // page] = 1 << 30
    f.meta.page_table = pt
    out, lse = f.decode(sliding_window=window)
    check(out, lse, ref, f"window {window} P{page}")
    assert pa.device_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (16, 16, 64), (24, 12, 128)])
@pytest.mark.parametrize("window", [1, 15, 333])
def test_window_ranges(cuda_device, hq, hkv, d, window):
    """Many sequences of which a window leaves little: ranges sized by the
    window, a workspace sized without it (the binding's)."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(51)
    L = rng.integers(1, 1500, 40).astype(np.int32)
    L[7] = 1
    p = W.small_problem(51, L - 1, np.ones_like(L), num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    f = FP4Problem(p, cuda_device, 52)
    ref = f.oracle(window=window)
    need = pa.decode_workspace_size(f.q.shape, f.k_cache, f.meta.max_seqlen_k, kv_dtype=pa.PA_KV_FP4, num_kv_heads=hkv)
    ws = torch.empty(need, dtype=torch.uint8, device=cuda_device)
    for kw in (dict(workspace=ws), dict(kv_chunk=32)):
        out, lse = f.decode(sliding_window=window, **kw)
        check(out, lse, ref, f"window {window} {hq}/{hkv} d{d} {list(kw)}")


@pytest.mark.parametrize("page_bad", [-1, 1 << 30])
def test_bad_page_between_head_groups(cuda_device, page_bad):
    """A page outside the pool where a row is several head groups: the error
    bit, and the other sequences right."""
    import paged_kv_flashattention_gb300 as pa
    L = np.array([50, 200, 90], np.int32)
    p = W.small_problem(53, L - 1, np.ones_like(L), num_q_heads=16, num_kv_heads=16, head_dim=128)
    f = FP4Problem(p, cuda_device, 54)
    ref = f.oracle()
    f.meta.page_table = f.meta.page_table.clone()
    f.meta.page_table[1, 3] = page_bad
    out, lse = f.decode()
    assert pa.device_error() == pa.PA_DEVERR_PAGE_RANGE
    keep = [0, 2]
    check(out[keep], lse[keep], tuple(x[keep] for x in ref), "beside a bad page")


def test_ragged_batch_d64(cuda_device):
    """64 sequences of U[128, 4096] keys, 32 / 8 heads of 64."""
    f = FP4Problem(W.config(2), cuda_device, 21)
    out, lse = f.decode()
    check(out, lse, f.oracle(), "ragged d64")


def test_long_contexts(cuda_device):
    rng = np.random.default_rng(31)
    L = np.exp(rng.uniform(np.log(512), np.log(16384), size=12)).astype(np.int32)
    p = W.small_problem(31, L - 1, np.ones_like(L), num_q_heads=32, num_kv_heads=8, head_dim=128)
    f = FP4Problem(p, cuda_device, 32)
    ref = f.oracle()
    for kw in (dict(), dict(max_ctas=7), dict(kv_chunk=4096)):
        out, lse = f.decode(**kw)
        check(out, lse, ref, f"long contexts {kw}")


def test_single_long_sequence_and_noalloc(cuda_device):
    import paged_kv_flashattention_gb300 as pa
    p = W.small_problem(33, [20010], [1], num_q_heads=32, num_kv_heads=8, head_dim=128, pool_factor=1.01)
    f = FP4Problem(p, cuda_device, 34)
    ref = f.oracle()
    out, lse = f.decode()
    check(out, lse, ref, "one long sequence")
    m = f.meta
    lse2 = torch.empty_like(lse)
    out2 = pa.decode_noalloc(f.q, f.k_cache, f.v_cache, m.page_table, m.cache_seqlens, m.max_seqlen_k, scale=p.scale,
                             lse=lse2, k_scale=f.k_scale, v_scale=f.v_scale, kv_dtype=pa.PA_KV_FP4)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_deterministic_and_page_order_free(cuda_device):
    """The same bits on every call, on a [slots, row bytes] pool, with a padded
    page table, and with the pages permuted in the pool."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(35)
    L = rng.integers(1, 900, 20).astype(np.int32)
    p = W.small_problem(35, L - 1, np.ones_like(L), num_q_heads=32, num_kv_heads=8, head_dim=128)
    f = FP4Problem(p, cuda_device, 36)
    out, lse = f.decode()
    o2, l2 = f.decode()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    m = f.meta
    flat = [c.view(-1, c.shape[-1]) for c in (f.k_cache, f.v_cache)]
    wide = torch.full((20, m.page_table.shape[1] + 9), 1 << 30, dtype=torch.int32, device=cuda_device)
    wide[:, :m.page_table.shape[1]] = m.page_table
    o3 = pa.decode(f.q, *flat, wide, m.cache_seqlens, m.max_seqlen_k, scale=p.scale, page_size=16, k_scale=f.k_scale,
                   v_scale=f.v_scale, kv_dtype=pa.PA_KV_FP4)
    assert torch.equal(out, o3)
    perm = torch.from_numpy(rng.permutation(p.num_pages)).to(cuda_device)
    inv = torch.argsort(perm).to(torch.int32)
    o4 = pa.decode(f.q, f.k_cache[perm].contiguous(), f.v_cache[perm].contiguous(), inv[m.page_table.long()].contiguous(),
                   m.cache_seqlens, m.max_seqlen_k, scale=p.scale, k_scale=f.k_scale, v_scale=f.v_scale,
                   kv_dtype=pa.PA_KV_FP4)
    assert torch.equal(out, o4)


def test_pool_past_32_bits(cuda_device):
    """Rows whose byte offsets pass 2^32: the last pages of a 4.6 GB pool."""
    import paged_kv_flashattention_gb300 as pa
    hkv, d, hq = 8, 128, 32
    rb = pa.fp4_row_bytes(hkv, d)
    pages = (9 << 29) // (16 * rb)
    rng = np.random.default_rng(37)
    lens = np.array([70, 33], np.int32)
    rows = random_rows(rng, 160, hkv, d)
    kc = torch.zeros((pages, 16, rb), dtype=torch.uint8, device=cuda_device)
    kc.view(-1, rb)[-160:] = dev_np(rows, cuda_device)
    pt = np.array([[pages - 1 - i for i in range(5)], [pages - 10 + i for i in range(5)]], np.int32)
    q = W.normal_bf16(rng, (2, hq, d))
    g = np.full(hkv, 0.004, np.float32)
    gd = dev_np(g, cuda_device)
    from pa_harness import bf16_dev
    lse = torch.empty((2, hq), dtype=torch.float32, device=cuda_device)
    out = pa.decode(bf16_dev(q, cuda_device), kc, kc, dev_np(pt, cuda_device), dev_np(lens, cuda_device), 80, lse=lse,
                    k_scale=gd, v_scale=gd, kv_dtype=pa.PA_KV_FP4)
    ref = fp4.attention(W.bf16_bits_to_f32(q), rows, rows, pt - (pages - 10), [0, 1, 2], [0, 70, 103], num_kv_heads=hkv,
                        page_size=16, k_scale=g, v_scale=g, scale=d ** -0.5)
    check(out, lse, ref, "pool past 32 bits")
    back, _ = pa.load_kv_fp4(torch.tensor([pages * 16 - 1], dtype=torch.int32, device=cuda_device), kc, kc, gd, gd, d)
    want = fp4.unpack(rows[-1:], hkv, d, g)
    assert np.abs(back.float().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max()


def test_bad_pages_and_lengths(cuda_device):
    """Page ids outside the pool are not read and raise the error bit, the
    other sequences are right; lengths past the bound are clamped."""
    import paged_kv_flashattention_gb300 as pa
    L = np.array([100, 64, 200], np.int32)
    p = W.small_problem(39, L - 1, np.ones_like(L), num_q_heads=16, num_kv_heads=4, head_dim=64)
    f = FP4Problem(p, cuda_device, 40)
    ref = f.oracle()
    pt = f.meta.page_table.clone()
    pt[1, 1], pt[1, 2] = -5, p.num_pages
    good, f.meta.page_table = f.meta.page_table, pt
    out, lse = f.decode()
    assert pa.device_error() == pa.PA_DEVERR_PAGE_RANGE
    keep = [0, 2]
    check(out[keep], lse[keep], tuple(x[keep] for x in ref), "beside a bad page")
    f.meta.page_table = good
    f.meta.cache_seqlens = dev_np(np.array([100, -3, 999], np.int32), cuda_device)
    out, lse = f.decode()
    assert pa.device_error() == pa.PA_DEVERR_SEQLENS
    want = [x.copy() for x in ref]
    want[0][1], want[1][1], want[2][1] = 0, -np.inf, 0
    check(out, lse, tuple(want), "clamped lengths")


def test_nan_scale_stays_in_its_head(cuda_device):
    """A block whose scale is NaN makes the heads that read it NaN, no other."""
    L = np.array([40, 40], np.int32)
    p = W.small_problem(41, L - 1, np.ones_like(L), num_q_heads=16, num_kv_heads=8, head_dim=128)
    f = FP4Problem(p, cuda_device, 42)
    ref = f.oracle()
    slot = int(p.token_table[0, 20])
    f.v_cache.view(-1, f.v_cache.shape[-1])[slot, 512 + 3 * 8 + 2] = 127      # head 3, block 2
    out, lse = f.decode()
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[0, 6:8, 32:48] = True
    assert torch.equal(bad, want)
    out = torch.where(bad, torch.from_numpy(ref[0]).to(out), out)
    check(out, lse, ref, "beside a NaN block")


@pytest.mark.parametrize("B", [1, 40])
def test_nan_key_reaches_the_output(cuda_device, B):
    """A key whose scale is NaN makes the rows that see it NaN, through both
    forms of the combine."""
    L = np.full(B, 600, np.int32)
    p = W.small_problem(45, L - 1, np.ones_like(L), num_q_heads=32, num_kv_heads=8, head_dim=128)
    f = FP4Problem(p, cuda_device, 46)
    slot = int(p.token_table[B - 1, 333])
    f.k_cache.view(-1, f.k_cache.shape[-1])[slot, 512 + 5 * 8] = 255          # head 5, block 0
    out, lse = f.decode()
    want = torch.zeros((B, 32), dtype=torch.bool, device=cuda_device)
    want[B - 1, 20:24] = True
    assert torch.equal(torch.isnan(out).all(-1), want) and torch.equal(torch.isnan(out).any(-1), want)
    assert torch.equal(torch.isnan(lse), want)


def test_captured_with_new_lengths(cuda_device):
    """One captured call serves other lengths and other rows; two graphs with
    their own workspaces run side by side."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(43)
    L = rng.integers(200, 1000, 9).astype(np.int32)
    p = W.small_problem(43, L - 1, np.ones_like(L), num_q_heads=32, num_kv_heads=8, head_dim=128)
    f = FP4Problem(p, cuda_device, 44)
    m = f.meta
    need = pa.decode_workspace_size(f.q.shape, f.k_cache, m.max_seqlen_k, kv_dtype=pa.PA_KV_FP4, num_kv_heads=8)
    runs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device=cuda_device)
        lens = m.cache_seqlens.clone()
        out, lse = torch.empty_like(f.q), torch.empty((9, 32), device=cuda_device)
        with torch.cuda.stream(s):
            def call():
                pa.decode(f.q, f.k_cache, f.v_cache, m.page_table, lens, m.max_seqlen_k, scale=p.scale, out=out, lse=lse,
                          workspace=ws, k_scale=f.k_scale, v_scale=f.v_scale, kv_dtype=pa.PA_KV_FP4)
            call()
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call()
        runs.append((g, lens, out, lse))
    short = (L * rng.uniform(0.1, 1.0, 9)).astype(np.int32).clip(1)
    runs[1][1].copy_(dev_np(short, cuda_device))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        runs[0][0].replay()
        with torch.cuda.stream(side):
            runs[1][0].replay()
    torch.cuda.synchronize()
    check(runs[0][2], runs[0][3], f.oracle(), "captured")
    from oracle_pins import _meta
    _, _, _, pt = _meta(p)
    ref = fp4.attention(W.bf16_bits_to_f32(p.q), f.kr, f.vr, pt, np.arange(10), np.concatenate([[0], np.cumsum(short)]),
                        num_kv_heads=8, page_size=16, k_scale=f.ks, v_scale=f.vs, scale=p.scale)
    check(runs[1][2], runs[1][3], ref, "captured, shorter")


def test_graph_runner(cuda_device):
    """Bucketed graphs over 4-bit pools: real rows right, dummies empty, and
    the same graph after the lengths change."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(45)
    L = rng.integers(1, 700, 20).astype(np.int32)
    p = W.small_problem(45, L - 1, np.ones_like(L), num_q_heads=16, num_kv_heads=4, head_dim=64)
    f = FP4Problem(p, cuda_device, 46)
    m = f.meta
    ref = f.oracle()
    runner = pa.DecodeGraphRunner(f.k_cache, f.v_cache, num_q_heads=16, max_seqlen_k=m.max_seqlen_k, buckets=(1, 8, 32),
                                  scale=p.scale, k_scale=f.k_scale, v_scale=f.v_scale, kv_dtype=pa.PA_KV_FP4, head_dim=64)
    runner.capture()
    for B in (3, 20, 1, 8):
        out, lse = runner.run(L[:B], q=f.q[:B], page_table=m.page_table[:B])
        torch.cuda.synchronize()
        check(out, lse, tuple(x[:B] for x in ref), f"graph B={B}")
        bucket = pa.bucket_for(runner.buckets, B)
        assert torch.count_nonzero(runner.out[B:bucket]).item() == 0
        assert torch.all(torch.isneginf(runner.lse[B:bucket]))
    short = (L * rng.uniform(0.1, 1.0, 20)).astype(np.int32).clip(1)
    out, lse = runner.run(short, q=f.q, page_table=m.page_table)
    torch.cuda.synchronize()
    from oracle_pins import _meta
    _, _, _, pt = _meta(p)
    ref = fp4.attention(W.bf16_bits_to_f32(p.q), f.kr, f.vr, pt, np.arange(21), np.concatenate([[0], np.cumsum(short)]),
                        num_kv_heads=4, page_size=16, k_scale=f.ks, v_scale=f.vs, scale=p.scale)
    check(out, lse, ref, "graph, shorter")


def test_many_sequences(cuda_device):
    """Thousands of short sequences, empty ones among them: more than a warp's
    or a CTA's share of the prefix."""
    rng = np.random.default_rng(57)
    L = rng.integers(1, 40, 4000).astype(np.int32)
    p = W.small_problem(57, L - 1, np.ones_like(L), num_q_heads=4, num_kv_heads=2, head_dim=64)
    f = FP4Problem(p, cuda_device, 58)
    empty = rng.random(4000) < 0.1
    lens = np.where(empty, 0, L).astype(np.int32)
    f.meta.cache_seqlens = dev_np(lens, cuda_device)
    out, lse = f.decode()
    want, want_l, mag = f.oracle()
    want[empty], want_l[empty], mag[empty] = 0, -np.inf, 0
    check(out, lse, (want, want_l, mag), "4000 sequences")
