"""The batch plan's free list with its place on the device: every page is given
out once over any number of calls and replays, against the oracle's loops with
the list moved on by hand."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_harness import dev_np
from oracle import batch as plan_oracle
from oracle import fp4
from test_batch_gpu import dev, table

pytestmark = pytest.mark.gpu

KEYS = ("cu_seqlens_q", "cu_seqlens_k", "cache_seqlens", "positions", "slot_mapping", "page_table", "totals")


@pytest.mark.parametrize("page", [1, 16, 7])
@pytest.mark.parametrize("B,hi_e", [(1, 9), (19, 3), (700, 40)])
def test_calls_in_a_row(cuda_device, page, B, hi_e):
    """Eager calls over one list until it runs out, every output each time."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(B + page)
    d, steps = cuda_device, 6
    start = rng.integers(0, 50, B)
    ext = rng.integers(0, hi_e + 1, (steps, B))
    max_k = int((start + ext.sum(0)).max()) + 1
    idx = rng.permutation(B)
    tt, free = table(rng, B, max_k, start, idx, page, spare=0)
    need = (-(-(start + ext.sum(0)) // page) - -(-start // page)).sum()
    free = (10 ** 5 + rng.permutation(int(need))).astype(np.int32)
    short = max(1, len(free) - 3)                    # the last calls find too few
    ttd, freed, cur = dev(tt, d), dev(free[:short], d), torch.zeros(2, dtype=torch.int32, device=d)
    pl = pa.BatchPlanner(d, B, int(ext.sum(1).max()) + 2, max_k, page)
    used, have, failed = 0, start.copy(), False
    for n in range(steps):
        before = pl.page_table.cpu().numpy()
        want = plan_oracle.build(have, ext[n], tt, idx, page, max_k, pl.max_tokens, before, free[used:short])
        b = pl.build(dev(have, d), dev(ext[n], d), ttd, dev(idx, d), free_pages=freed, free_cursor=cur)
        for k in KEYS:
            assert np.array_equal(getattr(b, k).cpu().numpy(), np.asarray(want[k])), f"call {n}: {k}"
        tt = want["token_table"]
        assert np.array_equal(ttd.cpu().numpy(), tt), f"call {n}: token table"
        used = min(used + want["totals"][3], short)
        assert cur.tolist() == [used, 0]
        bits = pa.device_error()
        assert bits == (pa.PA_DEVERR_NO_PAGES if "NO_PAGES" in want["error"] else 0)
        failed |= bits != 0
        have = have + ext[n]
        if failed:
            break
    assert failed == (short < need) and used == short


@pytest.mark.parametrize("bad", [-1, 9, 1 << 30])
def test_cursor_outside_the_list(cuda_device, bad):
    """Nothing is read outside the list: it counts as used up."""
    import paged_kv_flashattention_gb300 as pa
    d = cuda_device
    tt = torch.full((2, 40), 7, dtype=torch.int32, device=d)
    free = torch.arange(8, dtype=torch.int32, device=d)
    cur = torch.tensor([bad, 0], dtype=torch.int32, device=d)
    pl = pa.BatchPlanner(d, 2, 4, 40, 16)
    two, zero = torch.tensor([1, 3], dtype=torch.int32, device=d), torch.zeros(2, dtype=torch.int32, device=d)
    b = pl.build(zero, two, tt, torch.arange(2, dtype=torch.int32, device=d), free_pages=free, free_cursor=cur)
    assert pa.device_error() == pa.PA_DEVERR_NO_PAGES
    assert bool((b.slot_mapping == -1).all()) and bool((b.page_table[:, 0] == -1).all())
    assert cur.tolist() == [8, 0]


@pytest.mark.parametrize("planners", [1, 2])
def test_captured_steps(cuda_device, planners):
    """Sixty replays without a host read between them; with two planners (two
    halves of the requests) that take from one list in turn."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(7 + planners)
    d, B, page, max_k, steps = cuda_device, 24, 16, 400, 60
    start = rng.integers(0, 300, B)
    idx = rng.permutation(B)
    tt, free = table(rng, B, max_k, start, idx, page, spare=400)
    ttd, freed, cur = dev(tt, d), dev(free, d), torch.zeros(2, dtype=torch.int32, device=d)
    n = B // planners
    parts = []
    for i in range(planners):
        s = slice(i * n, (i + 1) * n)
        parts.append((pa.BatchPlanner(d, n, n, max_k, page), dev(start[s], d), torch.ones(n, dtype=torch.int32, device=d),
                      dev(idx[s], d)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for pl, cached, one, ix in parts:
                pl.build(cached, one, ttd, ix, free_pages=freed, free_cursor=cur)
                cached += 1
    for _ in range(steps):
        g.replay()
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    final, lens, seen = ttd.cpu().numpy(), start + steps, set()
    for r in range(B):
        row = final[idx[r], :lens[r]]
        assert np.array_equal(row[:start[r]], tt[idx[r], :start[r]])
        assert np.array_equal(row % page, np.arange(lens[r]) % page)
        pages = row[::page] // page
        assert np.all(row // page == pages.repeat(page)[:lens[r]])
        assert not seen & set(pages.tolist()), f"request {r} shares a page"
        seen |= set(pages.tolist())
    new = int((-(-lens // page) - -(-start // page)).sum())
    assert cur.tolist() == [new, 0]
    assert seen == set((tt[idx[r], j] // page) for r in range(B) for j in range(start[r])) | set(free[:new].tolist())


def test_the_readme_step(cuda_device):
    """README's step over a 4-bit cache, captured once and replayed across page
    boundaries; after every token each request's whole cache answers as its own
    history says."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(11)
    dv, B, hq, hkv, d, page, max_k, steps = cuda_device, 3, 8, 2, 64, 16, 64, 40
    start = np.array([0, 14, 16], np.int32)
    pages = 16
    rb = pa.fp4_row_bytes(hkv, d)
    k_cache = torch.full((pages, page, rb), 255, dtype=torch.uint8, device=dv)
    v_cache = k_cache.clone()
    gs = np.array([2e-3, 1.7e-3], np.float32)
    k_scale = v_scale = dev_np(gs, dv)
    order = rng.permutation(pages).astype(np.int32)
    token_table = torch.full((B, max_k), 1 << 30, dtype=torch.int32, device=dv)
    rows_k = [np.zeros((0, rb), np.uint8) for _ in range(B)]
    rows_v = [np.zeros((0, rb), np.uint8) for _ in range(B)]
    at = 0
    for b, n in enumerate(start):                    # the prompts, stored by the oracle
        if n:
            x, y = (W.bf16_bits_to_f32(W.normal_bf16(rng, (n, hkv, d))) for _ in range(2))
            rows_k[b], rows_v[b] = np.zeros((n, rb), np.uint8), np.zeros((n, rb), np.uint8)
            fp4.store(x, np.arange(n), rows_k[b], gs)
            fp4.store(y, np.arange(n), rows_v[b], gs)
            slots = order[at + np.arange(n) // page] * page + np.arange(n) % page
            at += -(-int(n) // page)
            token_table[b, :n] = dev(slots, dv)
            k_cache.view(-1, rb)[dev(slots, dv).long()] = dev_np(rows_k[b], dv)
            v_cache.view(-1, rb)[dev(slots, dv).long()] = dev_np(rows_v[b], dv)
    free_pages, cursor = dev(order[at:], dv), torch.zeros(2, dtype=torch.int32, device=dv)
    cached, one = dev(start, dv), torch.ones(B, dtype=torch.int32, device=dv)
    table_idx = torch.arange(B, dtype=torch.int32, device=dv)
    cos_sin = pa.rope_cos_sin_table(max_k, d).to(dv)
    q_in, k, v = (torch.zeros((B, h, d), dtype=torch.bfloat16, device=dv) for h in (hq, hkv, hkv))
    q = torch.empty_like(q_in)
    out, lse = torch.empty_like(q), torch.empty((B, hq), device=dv)
    plan = pa.BatchPlanner(dv, B, B, max_k, page)
    kv = dict(k_scale=k_scale, v_scale=v_scale, kv_dtype=pa.PA_KV_FP4)
    ws = torch.empty(pa.decode_workspace_size(q.shape, k_cache, max_k, kv_dtype=pa.PA_KV_FP4, num_kv_heads=hkv),
                     dtype=torch.uint8, device=dv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b = plan.build(cached, one, token_table, table_idx, free_pages=free_pages, free_cursor=cursor)
            pa.rope_store_kv(q_in, k, v, b.positions, cos_sin, b.slot_mapping, k_cache, v_cache, q_out=q, **kv)
            pa.decode(q, k_cache, v_cache, b.page_table, b.cache_seqlens, max_k, out=out, lse=lse, workspace=ws, **kv)
            cached += 1
    from fp4_harness import check
    for n in range(steps):
        for t in (q_in, k, v):
            t.copy_(torch.from_numpy(W.normal_bf16(rng, tuple(t.shape)).view(np.int16)).to(dv).view(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        # the stored row of each new token joins its request's own history
        slot = b.slot_mapping.cpu().numpy()
        now_k, now_v = k_cache.view(-1, rb).cpu().numpy(), v_cache.view(-1, rb).cpu().numpy()
        for r in range(B):
            rows_k[r] = np.concatenate([rows_k[r], now_k[slot[r]:slot[r] + 1]])
            rows_v[r] = np.concatenate([rows_v[r], now_v[slot[r]:slot[r] + 1]])
            ref = fp4.attention(q[r:r + 1].float().cpu().numpy(), rows_k[r], rows_v[r], np.arange(max_k)[None], [0, 1],
                                [0, len(rows_k[r])], num_kv_heads=hkv, page_size=1, k_scale=gs, v_scale=gs, scale=d ** -0.5)
            check(out[r:r + 1], lse[r:r + 1], ref, f"step {n} request {r}")
    assert pa.device_error() == 0
    assert cursor.tolist() == [int((-(-(start + steps) // page) - -(-start // page)).sum()), 0]
