"""GPU parity of prefill / extend over 4-bit pools against the fp64 oracle
(tolerances: fp4_harness), and the whole serving path over a 4-bit cache: plan,
rotary store, prefill, captured decode steps."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_harness import FP4Problem, check, dev_np
from oracle import fp4

pytestmark = pytest.mark.gpu

CASES = [
    ([0, 0, 0, 0, 0], [1, 15, 16, 17, 129]),
    ([3, 16, 127, 128, 1000], [1, 16, 1, 129, 255]),
    ([0, 7, 0], [300, 0, 128]),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 4), (32, 8), (6, 6), (8, 1), (24, 12), (32, 16)])
@pytest.mark.parametrize("page", [1, 16])
def test_edge_matrix(cuda_device, d, hq, hkv, page):
    import paged_kv_flashattention_gb300 as pa
    for n, (cached, ext) in enumerate(CASES):
        p = W.small_problem(500 + 7 * n + d + hq + page, cached, ext, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                            page_size=page)
        f = FP4Problem(p, cuda_device, n + hq)
        out, lse = f.prefill()
        check(out, lse, f.oracle(), f"d{d} {hq}/{hkv} P{page} case {n}")
    assert pa.device_error() == 0


@pytest.mark.parametrize("page", [1, 16])
def test_extend_partial_hit(cuda_device, page):
    """Eight requests over cached prefixes of up to 4096 keys."""
    p = W.config(4, "p1" if page == 1 else None)
    f = FP4Problem(p, cuda_device, 61)
    out, lse = f.prefill()
    check(out, lse, f.oracle(), f"extend P{page}")
    out2, lse2 = f.prefill(max_ctas=9)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_many_requests(cuda_device):
    """More requests than the class order takes: the order by tile number."""
    rng = np.random.default_rng(64)
    cached, ext = rng.integers(0, 200, 1500).astype(np.int32), rng.integers(0, 5, 1500).astype(np.int32)
    ext[700] = 260
    p = W.small_problem(64, cached, ext, num_q_heads=4, num_kv_heads=2, head_dim=64)
    f = FP4Problem(p, cuda_device, 65)
    check(*f.prefill(), f.oracle(), "1500 requests")


@pytest.mark.parametrize("extra", [0, 128, 5000, 300000])
def test_length_bound_above_the_lengths(cuda_device, extra):
    """max_seqlen_k is only a bound: the same bits whichever order of the work
    it leads to, requests without keys or rows among them."""
    p = W.small_problem(62, [0, 700, 0, 128, 127, 1, 0], [300, 128, 0, 256, 257, 1, 64], num_q_heads=8, num_kv_heads=4,
                        head_dim=128)
    f = FP4Problem(p, cuda_device, 63)
    m = f.meta
    check(*f.prefill(), f.oracle(), "exact bound")
    cols = -(-(m.max_seqlen_k + extra) // 16)
    wide = torch.full((7, cols), 1 << 30, dtype=torch.int32, device=cuda_device)
    wide[:, :m.page_table.shape[1]] = m.page_table
    m.page_table, m.max_seqlen_k = wide, m.max_seqlen_k + extra
    for kw in (dict(), dict(max_ctas=3)):
        check(*f.prefill(**kw), f.oracle(), f"bound + {extra} {kw}")


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [1, 17, 200])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (4, 4, 64)])
def test_windows(cuda_device, page, window, hq, hkv, d):
    p = W.small_problem(70 + window, [0, 300, 5], [200, 140, 1], num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page)
    f = FP4Problem(p, cuda_device, window)
    out, lse = f.prefill(sliding_window=window)
    check(out, lse, f.oracle(window=window), f"window {window} P{page}")


@pytest.mark.parametrize("page", [1, 16])
def test_block_mask_and_non_causal(cuda_device, page):
    """A block-sparse mask with empty rows, and attention without the causal
    limit."""
    cached, ext = [100, 0, 500], [300, 128, 250]
    rng = np.random.default_rng(80)
    p = W.small_problem(80, cached, ext, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=page)
    f = FP4Problem(p, cuda_device, 81)
    mask = W.block_mask(rng, ext, np.add(cached, ext), density=0.4, keep_diagonal=False)
    mask[1] = 0
    out, lse = f.prefill(block_mask=dev_np(mask, cuda_device))
    check(out, lse, f.oracle(block_mask=mask), f"block mask P{page}")
    p = W.small_problem(82, cached, ext, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=page, causal=False)
    f = FP4Problem(p, cuda_device, 83)
    out, lse = f.prefill()
    check(out, lse, f.oracle(), f"non-causal P{page}")


def test_bad_pages_and_lengths(cuda_device):
    """A page outside the pool reads as zeros and raises the error bit, a
    request past the bounds is skipped; the others are right."""
    import paged_kv_flashattention_gb300 as pa
    p = W.small_problem(90, [40, 64, 10], [60, 30, 100], num_q_heads=8, num_kv_heads=4, head_dim=128)
    for page_bad in (-7, p.num_pages):
        f = FP4Problem(p, cuda_device, 91)
        ref = f.oracle()
        f.meta.page_table = f.meta.page_table.clone()
        f.meta.page_table[1, 1] = page_bad
        out, lse = f.prefill()
        assert pa.device_error() == pa.PA_DEVERR_PAGE_RANGE
        keep = np.r_[0:60, 90:190]
        check(out[keep], lse[keep], tuple(x[keep] for x in ref), "beside a bad page")
    f = FP4Problem(p, cuda_device, 91)
    f.meta.cu_seqlens_k = dev_np(np.array([0, 100, 100 + 5000, 5210], np.int32), cuda_device)
    out, lse = f.prefill()
    assert pa.device_error() == pa.PA_DEVERR_SEQLENS
    check(out[keep], lse[keep], tuple(x[keep] for x in ref), "beside a skipped request")


def test_decode_equals_prefill_of_one_token(cuda_device):
    """Rows of one query through both kernels agree within the tolerances of
    both."""
    L = np.array([5, 130, 700, 1500], np.int32)
    p = W.small_problem(95, L - 1, np.ones_like(L), num_q_heads=32, num_kv_heads=8, head_dim=128)
    f = FP4Problem(p, cuda_device, 96)
    ref = f.oracle()
    for out, lse in (f.decode(), f.prefill()):
        check(out, lse, ref, "one token")


@pytest.mark.parametrize("fp4", [False, True])
def test_next_call_waits_for_an_overlapped_prefill(cuda_device, fp4):
    """A decode that runs beside a longer prefill, then calls that rewrite what
    the prefill reads (its page table; 4-bit rows): they come after it."""
    import paged_kv_flashattention_gb300 as pa
    from pa_harness import bf16_dev
    dev = cuda_device
    p = W.small_problem(98, [3000, 2000], [600, 500], num_q_heads=16, num_kv_heads=4, head_dim=128)
    f = FP4Problem(p, dev, 99)
    m = f.meta
    kw = dict(scale=p.scale)
    kc, vc = f.k_cache, f.v_cache
    if fp4:
        kw.update(k_scale=f.k_scale, v_scale=f.v_scale, kv_dtype=pa.PA_KV_FP4)
    else:
        kc, vc = (torch.randn((p.num_pages, 16, 4, 128), device=dev).to(torch.bfloat16) for _ in range(2))
    args = (m.cu_seqlens_q, m.cu_seqlens_k, m.max_seqlen_q, m.max_seqlen_k)
    want = pa.prefill(f.q, kc, vc, m.page_table, *args, **kw)
    qd = bf16_dev(W.normal_bf16(np.random.default_rng(1), (2, 16, 128)), dev)
    lens = torch.tensor([40, 70], dtype=torch.int32, device=dev)
    table = m.page_table.clone()
    ws = torch.empty(max(16, pa.decode_workspace_size(qd.shape, kc, 80, **({"kv_dtype": pa.PA_KV_FP4, "num_kv_heads": 4}
                                                                         if fp4 else {}))), dtype=torch.uint8, device=dev)
    # a plan whose page table is the one the prefill reads
    pl = pa.BatchPlanner(dev, 2, 2, m.max_seqlen_k, 16)
    pl.page_table[:2, :table.shape[1]] = table
    tt = torch.zeros((2, m.max_seqlen_k), dtype=torch.int32, device=dev)
    idx = torch.arange(2, dtype=torch.int32, device=dev)
    one = torch.ones(2, dtype=torch.int32, device=dev)
    slots = torch.arange(64, dtype=torch.int32, device=dev)
    k = torch.ones((64, 4, 128), dtype=torch.bfloat16, device=dev)
    out, out_d = torch.empty_like(f.q), torch.empty_like(qd)
    torch.cuda.synchronize()
    pa.prefill(f.q, kc, vc, pl.page_table[:2], *args, out=out, max_ctas=4, **kw)
    pa.decode(qd, kc, vc, table, lens, 80, out=out_d, workspace=ws, overlap_previous=True, max_ctas=64, **kw)
    pl.build(one * (m.max_seqlen_k - 1), one, tt, idx)
    if fp4:
        pa.store_kv_fp4(k, k, slots, kc, vc, f.k_scale, f.v_scale)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert int(pl.page_table[:2, :table.shape[1]].abs().sum()) == 0, "the plan was built"


@pytest.mark.parametrize("page,hq,hkv,d", [(16, 32, 8, 128), (1, 8, 2, 64)])
def test_serving_over_a_4bit_cache(cuda_device, page, hq, hkv, d):
    """The operators together: the plan gives new prompts their pages, the
    rotary store writes the cache, prefill answers; then captured decode steps
    (plan, rotary store, decode) whose lengths live on the device."""
    import paged_kv_flashattention_gb300 as pa
    dev = cuda_device
    rng = np.random.default_rng(97)
    B, max_k, steps = 4, 320, 3
    first = np.array([33, 1, 200, 120], np.int32)
    idx = np.array([2, 0, 3, 1], np.int32)
    pages = 4 * (max_k // page + 1) + 3
    free = rng.permutation(pages).astype(np.int32)
    rb = pa.fp4_row_bytes(hkv, d)
    kc = torch.full((pages, page, rb), 255, dtype=torch.uint8, device=dev)
    vc = kc.clone()
    g = np.linspace(1.5e-3, 2.5e-3, hkv).astype(np.float32)
    gd = dev_np(g, dev)
    cs = pa.rope_cos_sin_table(max_k, d).to(dev)
    tt = torch.full((B, max_k), 1 << 30, dtype=torch.int32, device=dev)
    idxd, freed = dev_np(idx, dev), dev_np(free, dev)
    history = [[] for _ in range(B)]                 # per request: (q, k, v) of every token, bf16 bits

    def draw(n):
        return [torch.from_numpy(W.normal_bf16(rng, (n, h, d)).view(np.int16)).to(dev).view(torch.bfloat16)
                for h in (hq, hkv, hkv)]

    def oracle_for(lens_now, extend):
        """fp64 attention over what the cache stands for after a step."""
        rows = [c.view(-1, rb).cpu().numpy() for c in (kc, vc)]
        cu_q = np.concatenate([[0], np.cumsum(extend)])
        cu_k = np.concatenate([[0], np.cumsum(lens_now)])
        table = tt.cpu().numpy()[idx]
        return rows, table, cu_q, cu_k

    total = int(first.sum())
    plan = pa.BatchPlanner(dev, B, total + 5, max_k, page)
    zero, ext = torch.zeros(B, dtype=torch.int32, device=dev), dev_np(first, dev)
    b = plan.build(zero, ext, tt, idxd, free_pages=freed)
    q, k, v = draw(total + 5)                        # five rows of padding
    q = pa.rope_store_kv(q, k, v, b.positions, cs, b.slot_mapping, kc, vc, k_scale=gd, v_scale=gd, kv_dtype=pa.PA_KV_FP4)
    out = torch.full_like(q, 7.0)
    lse = torch.zeros((hq, total + 5), device=dev)
    pa.prefill(q, kc, vc, b.page_table, b.cu_seqlens_q, b.cu_seqlens_k, int(first.max()), max_k, page_size=page, out=out,
               lse=lse, k_scale=gd, v_scale=gd, kv_dtype=pa.PA_KV_FP4)
    assert pa.device_error() == 0
    assert bool((out[total:] == 7).all()), "rows behind the last sequence were written"
    rows, table, cu_q, cu_k = oracle_for(first, first)
    qf = q[:total].float().cpu().numpy()
    ref = fp4.attention(qf, rows[0], rows[1], table, cu_q, cu_k, num_kv_heads=hkv, page_size=1, k_scale=g, v_scale=g,
                        scale=d ** -0.5)
    check(out[:total], lse[:, :total].t(), ref, "prefill over the plan's pages")
    # the cache holds the rotated keys: row by row what the store's oracle gives
    want = np.full(rows[0].shape, 255, np.uint8)
    fp4.store(v[:total].float().cpu().numpy(), b.slot_mapping.cpu().numpy()[:total], want, g)
    assert np.array_equal(want, rows[1])

    used = int(b.totals[3])
    cached, one = dev_np(first, dev), torch.ones(B, dtype=torch.int32, device=dev)
    step_plan = pa.BatchPlanner(dev, B, B, max_k, page)
    nextfree = freed[used:used + B].clone()
    qs, ks, vs = draw(B)
    qr, o, ls = torch.empty_like(qs), torch.empty_like(qs), torch.empty((B, hq), device=dev)
    need = pa.decode_workspace_size(qs.shape, kc, max_k, kv_dtype=pa.PA_KV_FP4, num_kv_heads=hkv)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def step():
        sb = step_plan.build(cached, one, tt, idxd, free_pages=nextfree)
        pa.rope_store_kv(qs, ks, vs, sb.positions, cs, sb.slot_mapping, kc, vc, q_out=qr, k_scale=gd, v_scale=gd,
                         kv_dtype=pa.PA_KV_FP4)
        pa.decode(qr, kc, vc, sb.page_table, sb.cache_seqlens, max_k, out=o, lse=ls, workspace=ws, k_scale=gd, v_scale=gd,
                  kv_dtype=pa.PA_KV_FP4)
        return sb

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = (tt.clone(), kc.clone(), vc.clone())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sb = step()
    for t, x in zip((tt, kc, vc), keep):
        t.copy_(x)
    lens = first.copy()
    for n in range(steps):
        for t, x in zip((qs, ks, vs), draw(B)):
            t.copy_(x)
        nextfree.copy_(freed[used:used + B])
        graph.replay()
        torch.cuda.synchronize()
        lens += 1
        used += int(sb.totals[3])
        rows, table, cu_q, cu_k = oracle_for(lens, np.ones(B, int))
        ref = fp4.attention(qr.float().cpu().numpy(), rows[0], rows[1], table, cu_q, cu_k, num_kv_heads=hkv, page_size=1,
                            k_scale=g, v_scale=g, scale=d ** -0.5)
        check(o, ls, ref, f"decode step {n}")
        cached += 1
    assert pa.device_error() == 0
    assert used == sum(-(-int(n) // page) for n in lens)
