"""The batch plan built on the GPU against the oracle's loops, every output
element, and against the host metadata path."""
import numpy as np
import pytest
import torch

import oracle
from oracle import batch as plan_oracle

pytestmark = pytest.mark.gpu


def dev(a, d):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(d)


def table(rng, rows, width, lens, idx, page, spare=500):
    """A token table whose requests lie on random pages, and the pages that are
    free; entries past a request's length hold 10^9."""
    need = [-(-n // page) for n in lens]
    perm = rng.permutation(sum(need) + spare)
    tt = np.full((rows, width), 10 ** 9, np.int32)
    at = 0
    for b, n in enumerate(lens):
        pages = perm[at:at + need[b]]
        at += need[b]
        j = np.arange(n)
        if 0 <= idx[b] < rows:
            tt[idx[b], :n] = pages[j // page] * page + j % page
    return tt, perm[at:].astype(np.int32)


def run(d, cached, extend, tt, idx, page, max_k, tokens, free=None, planner=None):
    import paged_kv_flashattention_gb300 as pa
    pl = planner or pa.BatchPlanner(d, len(cached) + 3, tokens, max_k, page)
    ttd = dev(tt, d)
    before = pl.page_table.cpu().numpy()[:len(cached)]
    b = pl.build(dev(cached, d), dev(extend, d), ttd, dev(idx, d), free_pages=None if free is None else dev(free, d))
    got = {k: getattr(b, k).cpu().numpy() for k in ("cu_seqlens_q", "cu_seqlens_k", "cache_seqlens", "positions",
                                                    "slot_mapping", "page_table", "totals")}
    got["token_table"] = ttd.cpu().numpy()
    bits = pa.device_error()
    want = plan_oracle.build(cached, extend, tt, idx, page, max_k, tokens, before, free)
    for k, v in got.items():
        w = np.asarray(want[k])
        bad = np.argwhere(v != w)
        assert v.shape == w.shape and bad.size == 0, f"{k}: {len(bad)} of {w.size} differ, first at {bad[:1]}"
    names = {n: getattr(pa, f"PA_DEVERR_{n}") for n in ("SEQLENS", "TABLE_INDEX", "NO_PAGES")}
    assert bits == sum(names[n] for n in want["error"])
    return b, got, pl


@pytest.mark.parametrize("page", [1, 16, 7])
@pytest.mark.parametrize("take", [False, True])
@pytest.mark.parametrize("B,hi_c,hi_e,slack", [(0, 0, 0, 5), (1, 0, 1, 0), (1, 33, 700, 3), (5, 40, 40, 0), (256, 300, 1, 0),
                                               (300, 50, 9, 100), (1100, 20, 3, 1)])
def test_against_loops(cuda_device, page, take, B, hi_c, hi_e, slack):
    rng = np.random.default_rng(B * 100 + page + hi_e)
    cached = rng.integers(0, hi_c + 1, B)
    extend = rng.integers(0 if B > 1 else hi_e, hi_e + 1, B)
    lens = cached + extend
    max_k = int(lens.max()) + 2 if B else 4
    idx = rng.permutation(B + 4)[:B]
    tt, free = table(rng, B + 4, max_k + 3, cached if take else lens, idx, page, spare=int(extend.sum()) + 8)
    run(cuda_device, cached, extend, tt, idx, page, max_k, int(extend.sum()) + slack, free if take else None)


def test_broken_requests(cuda_device):
    """Negative and too long lengths, rows outside the table, too few tokens
    and too few free pages: each raises its bit and leaves the rest right."""
    rng = np.random.default_rng(3)
    page, max_k = 16, 100
    cached = np.array([10, -1, 90, 40, 50, 16])
    extend = np.array([20, 5, 11, 20, -2, 33])
    idx = np.array([3, 1, 0, 9, 2, 5])
    tt, free = table(rng, 6, max_k, [10, 0, 90, 0, 0, 16], idx, page)
    run(cuda_device, cached, extend, tt, idx, page, max_k, 80, free)
    run(cuda_device, cached, extend, tt, idx, page, max_k, 30, free)      # tokens past the end
    run(cuda_device, cached, extend, tt, idx, page, max_k, 80, free[:2])  # the list runs out
    run(cuda_device, cached, extend, tt, idx, page, max_k, 80, free[:0])  # no page at all
    idx[3] = -1
    run(cuda_device, cached, extend, tt, idx, page, max_k, 80)


def test_matches_the_host_path(cuda_device):
    """The same boundaries and page table as the host metadata, and shared
    table rows (prefix sharing) without a free list."""
    import paged_kv_flashattention_gb300 as pa
    from paged_kv_flashattention_gb300 import metadata
    rng = np.random.default_rng(5)
    cached, extend = rng.integers(0, 400, 30), rng.integers(0, 60, 30)
    lens = cached + extend
    idx = rng.permutation(32)[:30]
    tt, _ = table(rng, 32, 500, lens, idx, 16)
    b, got, _ = run(cuda_device, cached, extend, tt, idx, 16, int(lens.max()), int(extend.sum()))
    m = metadata.prepare(cached, extend, dev(tt, cuda_device), dev(idx, cuda_device), 16)
    assert torch.equal(m.cu_seqlens_q, b.cu_seqlens_q) and torch.equal(m.cu_seqlens_k, b.cu_seqlens_k)
    assert torch.equal(m.cache_seqlens, b.cache_seqlens)
    for r, n in enumerate(lens):
        c = -(-int(n) // 16)
        assert torch.equal(m.page_table[r, :c], b.page_table[r, :c])
    want = oracle.seqlens(cached, extend)
    assert tuple(got["totals"][1:3]) == tuple(want[3:5])
    idx[:] = idx[0]
    run(cuda_device, np.minimum(cached, 5), np.minimum(extend, 5), tt, idx, 16, int(lens.max()), 200)


def test_decode_steps_in_a_graph(cuda_device):
    """Forty captured steps: each request grows by one token, pages are taken
    as they fill up, and the table holds every slot at the end."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(7)
    B, page, max_k, steps = 19, 16, 400, 40
    start = rng.integers(0, 300, B)
    idx = rng.permutation(B)
    tt, free = table(rng, B, max_k, start, idx, page, spare=400)
    d = cuda_device
    ttd, idxd, freed = dev(tt, d), dev(idx, d), dev(free, d)
    cached, ones = dev(start, d), torch.ones(B, dtype=torch.int32, device=d)
    pl = pa.BatchPlanner(d, B, B, max_k, page)
    window = freed[:B].clone()                       # the list's next entries, refreshed between steps
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = ttd.clone()
    with torch.cuda.stream(s):
        pl.build(cached, ones, ttd, idxd, free_pages=window)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b = pl.build(cached, ones, ttd, idxd, free_pages=window)
    ttd.copy_(keep)
    used, seen = 0, []
    for step in range(steps):
        window.copy_(freed[used:used + B])
        g.replay()
        torch.cuda.synchronize()
        n = int(b.totals[3])
        seen.append(b.slot_mapping.cpu().numpy().copy())
        used += n
        cached += 1
    assert pa.device_error() == 0
    final = ttd.cpu().numpy()
    table_slots = set()
    for r in range(B):
        n = int(start[r]) + steps
        row = final[idx[r], :n]
        assert np.array_equal(row[:start[r]], tt[idx[r], :start[r]])
        assert np.array_equal(row[start[r]:], [x[r] for x in seen])
        assert np.array_equal(row % page, np.arange(n) % page)
        assert np.all(row // page == (row[::page] // page).repeat(page)[:n])
        table_slots |= set(row.tolist())
    assert len(table_slots) == int((start + steps).sum())
    assert used == sum(-(-(int(a) + steps) // page) - -(-int(a) // page) for a in start)


def test_many_requests(cuda_device):
    """16384 requests, the largest batch."""
    rng = np.random.default_rng(8)
    B = 16384
    cached, extend = rng.integers(0, 20, B), rng.integers(0, 3, B)
    idx = rng.permutation(B)
    tt, free = table(rng, B, 24, cached, idx, 16, spare=B)
    run(cuda_device, cached, extend, tt, idx, 16, 24, int(extend.sum()), free)
