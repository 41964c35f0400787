"""Beam search's selection and the reordering of paged states, against plain
implementations on the host in 64 bits.

Selection: beams and tokens are exact; a total is one rounding to fp32 (2^-24 of
itself) off, and lse's error, below 2^-20 (see csrc/beam.cu), which is far from
any two totals of these inputs unless they are equal.  Reordering moves bits.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

NEG = float("-inf")


def plain_select(logits, scores, n, finished=None, pad=0):
    """logits fp64 [G * K, V] -> (totals, parents, tokens), each [G, n]."""
    x = np.where(np.isnan(logits) | (logits == np.inf), NEG, logits)
    sc = np.where(np.isnan(scores) | (scores == np.inf), NEG, scores).astype(np.float64)
    G, K = sc.shape
    V = x.shape[1]
    with np.errstate(invalid="ignore", divide="ignore"):
        top = x.max(1, keepdims=True)
        top = np.where(np.isinf(top), 0.0, top)
        lse = top + np.log(np.exp(x - top).sum(1, keepdims=True))
        total = sc.reshape(-1, 1) + (x - lse)
    total = np.where(np.isnan(total), NEG, total).reshape(G, K, V)
    if finished is not None:
        for g, k in zip(*np.nonzero(finished)):
            total[g, k] = NEG
            total[g, k, pad] = sc[g, k]
    total = total.reshape(G, K * V)
    at = np.argsort(-total, axis=1, kind="stable")[:, :n]
    return np.take_along_axis(total, at, 1), at // V, at % V


def check_select(dev, logits, scores, n, finished=None, pad=0, **kw):
    import paged_kv_flashattention_gb300 as pa
    got = pa.beam_select(logits, scores, n, finished=finished, pad_token=pad, **kw)
    G, K = scores.shape
    x = logits.reshape(G * K, logits.shape[-1]).double().cpu().numpy()
    want = plain_select(x, scores.cpu().numpy(), n, None if finished is None else finished.cpu().numpy(), pad)
    assert pa.device_error() == 0
    assert np.array_equal(got[1].cpu().numpy(), want[1]), "parents"
    assert np.array_equal(got[2].cpu().numpy(), want[2]), "tokens"
    t = got[0].double().cpu().numpy()
    fin = np.isfinite(want[0])
    assert np.array_equal(np.isfinite(t), fin) and bool((t[~fin] == NEG).all())
    assert fin.sum() == 0 or bool((np.abs(t - want[0])[fin] <= 2.0 ** -24 * np.abs(want[0][fin]) + 2.0 ** -20).all())
    return got


def logits_of(dev, rows, V, dtype, seed, spread=3.0, slack=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((rows, V + slack), generator=g, device=dev) * spread
    x[:, V:] = float("nan")
    return x.to(dtype)[:, :V]


def scores_of(dev, G, K, seed):
    g = torch.Generator(device=dev).manual_seed(seed + 1000)
    return -20 * torch.rand((G, K), generator=g, device=dev)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V,slack", [(1, 0), (7, 0), (8, 3), (33, 0), (2047, 1), (2048, 0), (2049, 0), (5000, 7), (32000, 0), (50257, 0),
                                     (50257, 5), (128256, 0)])
def test_vocabularies(cuda_device, V, slack, dtype):
    """Odd sizes and row distances: every alignment of a row's start."""
    for G, K, n in ((1, 1, 1), (3, 3, 4), (2, 5, 10)):
        n = min(n, V)
        check_select(cuda_device, logits_of(cuda_device, G * K, V, dtype, V + K, slack=slack), scores_of(cuda_device, G, K, V), n)


@pytest.mark.parametrize("G,K,n", [(1, 64, 128), (4, 16, 32), (70, 4, 8), (1, 2, 128), (300, 1, 3), (9, 7, 65)])
def test_counts(cuda_device, G, K, n):
    check_select(cuda_device, logits_of(cuda_device, G * K, 9001, torch.bfloat16, K), scores_of(cuda_device, G, K, n), n)


def test_three_dimensions_and_defaults(cuda_device):
    import paged_kv_flashattention_gb300 as pa
    x = logits_of(cuda_device, 12, 1000, torch.float32, 1)
    s = scores_of(cuda_device, 3, 4, 1)
    a = pa.beam_select(x, s)
    b = pa.beam_select(x.view(3, 4, 1000), s)
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and a[0].shape == (3, 4)
    c = pa.beam_select(x, s.clone(), 4, out_scores=s)            # scores in place
    assert c[0] is s and torch.equal(s, a[0])


@pytest.mark.parametrize("n", [1, 8, 128])
def test_equal_logits(cuda_device, n):
    """All logits equal (every tile is full of candidates), and equal beams."""
    x = torch.zeros((6, 20000), dtype=torch.bfloat16, device=cuda_device)
    check_select(cuda_device, x, torch.zeros((2, 3), device=cuda_device), n)
    x[:, ::2] = -0.0
    check_select(cuda_device, x, torch.zeros((2, 3), device=cuda_device), n)
    y = logits_of(cuda_device, 1, 30011, torch.float32, 4).expand(6, -1).contiguous()      # rows of every alignment
    check_select(cuda_device, y, torch.full((2, 3), -1.5, device=cuda_device), n)
    y = logits_of(cuda_device, 1, 30011, torch.bfloat16, 5).expand(8, -1).contiguous()
    check_select(cuda_device, y, torch.full((1, 8), -1.5, device=cuda_device), n)


@pytest.mark.parametrize("how", ["rising", "falling", "steps", "peak_last"])
@pytest.mark.parametrize("n", [4, 64])
def test_orders(cuda_device, how, n):
    """Rising rows put every element above the threshold that came before it."""
    V = 40000
    i = torch.arange(V, device=cuda_device, dtype=torch.float32)
    row = {"rising": i * 1e-3, "falling": -i * 1e-3, "steps": torch.floor(i / 1000) * 0.125,
           "peak_last": torch.where(i == V - 1, 50.0, 0.0)}[how]
    x = torch.stack([row, row * 0.5, row.flip(0)])
    check_select(cuda_device, x, scores_of(cuda_device, 1, 3, n), n)
    check_select(cuda_device, x * 100, scores_of(cuda_device, 1, 3, n), n)        # spread of thousands


def test_chance_order_does_not_matter(cuda_device):
    """The same call gives the same bits."""
    import paged_kv_flashattention_gb300 as pa
    x = (torch.arange(70000, device=cuda_device) % 4099).float().repeat(8, 1) * 0.003
    s = scores_of(cuda_device, 2, 4, 0)
    ref = pa.beam_select(x, s, 100)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(ref, pa.beam_select(x, s, 100)))


@pytest.mark.parametrize("keep", [0, 1, 3, 60])
@pytest.mark.parametrize("n", [1, 6, 64])
def test_banned_words(cuda_device, keep, n):
    """Rows of which a few words are left, or none; NaN and +inf among them."""
    G, K, V = 3, 4, 9000
    x = logits_of(cuda_device, G * K, V, torch.float32, keep)
    g = torch.Generator(device=cuda_device).manual_seed(keep)
    at = torch.argsort(torch.rand(x.shape, generator=g, device=cuda_device), 1)
    mask = torch.ones_like(x, dtype=torch.bool)
    mask.scatter_(1, at[:, :keep], False)
    x = x.masked_fill(mask, NEG)
    x[1, 5], x[2, 7], x[3, :] = float("nan"), float("inf"), NEG
    check_select(cuda_device, x, scores_of(cuda_device, G, K, keep), n)
    check_select(cuda_device, torch.full_like(x, NEG), scores_of(cuda_device, G, K, keep), n)
    # the type's lowest value is a value
    low = torch.full((4, 3000), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device=cuda_device)
    low[:, 100] = 1.0
    check_select(cuda_device, low, scores_of(cuda_device, 1, 4, keep), n)


@pytest.mark.parametrize("pad", [0, 3, 699])
@pytest.mark.parametrize("n", [1, 5, 64])
def test_finished_and_dead_beams(cuda_device, pad, n):
    G, K, V = 4, 5, 700
    x = logits_of(cuda_device, G * K, V, torch.bfloat16, pad)
    s = scores_of(cuda_device, G, K, n)
    f = torch.zeros((G, K), dtype=torch.uint8, device=cuda_device)
    f[0, 1] = f[1] = 1
    f[2, 0] = 7
    s[0, 0], s[2, 0], s[2, 3], s[3] = NEG, float("nan"), float("inf"), NEG
    x[5:10] = float("nan")                               # logits of ended beams are not read
    check_select(cuda_device, x, s, n, f, pad)
    check_select(cuda_device, x, s, n, f.bool(), pad)


def test_first_step(cuda_device):
    """Beams that start alike: all but the first at -inf."""
    x = logits_of(cuda_device, 1, 32000, torch.bfloat16, 3).expand(4, -1).contiguous()
    s = torch.tensor([[0.0, NEG, NEG, NEG]], device=cuda_device)
    got = check_select(cuda_device, x, s, 4)
    assert got[1].tolist() == [[0, 0, 0, 0]]


def test_select_captured_and_shared_workspace(cuda_device):
    import paged_kv_flashattention_gb300 as pa
    x = logits_of(cuda_device, 8, 6000, torch.bfloat16, 1)
    s = scores_of(cuda_device, 2, 4, 1)
    outs = [torch.empty((2, 4), dtype=t, device=cuda_device) for t in (torch.float32, torch.int32, torch.int32)]
    ws = torch.empty(pa.beam_select_workspace_size(2, 4, 6000, 4), dtype=torch.uint8, device=cuda_device)

    def call():
        pa.beam_select(x, s, 4, out_scores=outs[0], parents=outs[1], tokens=outs[2], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        torch.cuda.synchronize()
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]      # two graphs that share the workspace
        for graph in graphs:
            with torch.cuda.graph(graph, stream=side):
                call()
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(logits_of(cuda_device, 8, 6000, torch.bfloat16, 50 + i))
        ws.fill_(255)
        graphs[i % 2].replay()
        want = plain_select(x.double().cpu().numpy(), s.cpu().numpy(), 4)
        assert np.array_equal(outs[1].cpu().numpy(), want[1]) and np.array_equal(outs[2].cpu().numpy(), want[2])


# ------------------------------------------------------------- reordering
def plain_reorder(parents, table, idx, lens, spare, pools, page, first=None, history=None):
    """numpy, in place; pools [pages, page, row bytes]."""
    G, K = parents.shape
    old_t, old_s = table.copy(), spare.copy()
    old_p = [p.copy() for p in pools]
    old_h = None if history is None else history.copy()
    for g in range(G):
        for i in range(K):
            me, q = g * K + i, g * K + parents[g, i]
            if q == me:
                continue
            L = int(lens[me])
            part = L % page
            lo = 0 if first is None else int(first[me])
            table[idx[me], lo:L - part] = old_t[idx[q], lo:L - part]
            if part:
                src, dst = old_t[idx[q], L - 1] // page, old_s[me]
                for p, o in zip(pools, old_p):
                    p[dst, :part] = o[src, :part]
                table[idx[me], L - part:L] = dst * page + np.arange(part)
                spare[me] = old_t[idx[me], L - 1] // page
            if history is not None:
                history[me] = old_h[q]


def reorder_case(rng, G, K, page, longest, pages_extra=3, layers=2, row=(2, 64), dtype=torch.bfloat16):
    N = G * K
    lens = np.repeat(rng.integers(0, longest + 1, G), K).astype(np.int32)
    need = -(-lens // page)
    ids = rng.permutation(int(need.sum()) + N + pages_extra).astype(np.int32)
    spare, ids = ids[:N].copy(), list(ids[N:])
    rows = N + 2
    table = np.full((rows, longest + 5), -7, np.int32)
    idx = rng.permutation(rows)[:N].astype(np.int32)
    for i in range(N):
        for c in range(need[i]):
            p = ids.pop()
            j = np.arange(c * page, min((c + 1) * page, lens[i]))
            table[idx[i], j] = p * page + j % page
    n = int(need.sum()) + N + pages_extra
    pools = [torch.from_numpy(rng.integers(0, 256, (n, page) + row[:-1] + (row[-1] * (2 if dtype == torch.bfloat16 else 1),), dtype=np.uint8))
             for _ in range(2 * layers)]
    parents = rng.integers(0, K, (G, K)).astype(np.int32)
    return parents, table, idx, lens, spare, pools, dtype


def run_reorder(dev, case, page, first=None, history=None, **kw):
    import paged_kv_flashattention_gb300 as pa
    parents, table, idx, lens, spare, pools, dtype = case
    d = lambda a: None if a is None else torch.from_numpy(np.array(a)).to(dev)
    dp = [p.to(dev).view(dtype) if dtype != torch.uint8 else p.to(dev) for p in pools]
    t, s, h = d(table), d(spare), d(history)
    half = len(dp) // 2
    pa.beam_reorder(d(parents), t, d(idx), d(lens), s, dp[:half], dp[half:], prefix_lens=d(first), history=h, **kw)
    want = [p.flatten(2).numpy().copy() for p in pools]
    table, spare = table.copy(), spare.copy()
    history = None if history is None else history.copy()
    plain_reorder(parents, table, idx, lens, spare, want, page, first, history)
    assert np.array_equal(t.cpu().numpy(), table), "token table"
    assert np.array_equal(s.cpu().numpy(), spare), "spare pages"
    for p, w in zip(dp, want):
        assert np.array_equal(p.view(torch.uint8).flatten(2).cpu().numpy(), w), "pool"
    if history is not None:
        assert np.array_equal(h.cpu().numpy(), history), "history"


@pytest.mark.parametrize("G,K", [(1, 1), (1, 2), (3, 4), (2, 5), (1, 64), (40, 8)])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("longest", [0, 1, 17, 127, 400])
def test_reorder(cuda_device, G, K, page, longest):
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(G * 100 + K + longest)
    case = reorder_case(rng, G, K, page, longest)
    run_reorder(cuda_device, case, page)
    history = rng.integers(0, 9999, (G * K, 301)).astype(np.int32)
    first = np.minimum(case[3], 33 // page * page).astype(np.int32)
    # slots below the prefix are the same in a group's rows
    parents, table, idx, lens = case[:4]
    for i in range(G * K):
        table[idx[i], :first[i]] = table[idx[i // K * K], :first[i]]
    run_reorder(cuda_device, case, page, first=first, history=history)
    assert pa.device_error() == 0


@pytest.mark.parametrize("dtype,row", [(torch.uint8, (2, 64)), (torch.uint8, (144,)), (torch.bfloat16, (8, 128)), (torch.bfloat16, (1, 8))])
def test_reorder_pools(cuda_device, dtype, row):
    """FP8 and 4-bit rows, large and small ones, many pools."""
    rng = np.random.default_rng(5)
    run_reorder(cuda_device, reorder_case(rng, 2, 4, 16, 60, layers=5, row=row, dtype=dtype), 16)
    run_reorder(cuda_device, reorder_case(rng, 2, 4, 16, 60, layers=1, row=row, dtype=dtype), 16)


def test_reorder_every_remainder_and_parents(cuda_device):
    """Lengths of every remainder; cycles, all from one, none moved."""
    rng = np.random.default_rng(6)
    for L in range(120, 137):
        case = list(reorder_case(rng, 1, 6, 16, 140))
        case = list(reorder_case(rng, 3, 6, 16, L))
        keep = case[3]
        case[0] = np.array([[1, 2, 3, 4, 5, 0], [2, 2, 2, 2, 2, 2], [0, 1, 2, 3, 4, 5]], np.int32)
        assert keep.max() <= L
        run_reorder(cuda_device, tuple(case), 16)


def test_reorder_bad_device_data(cuda_device):
    """Groups that the bad entry does not concern move as they should."""
    import paged_kv_flashattention_gb300 as pa
    rng = np.random.default_rng(8)
    for what in ("parent", "negative_parent", "idx", "length", "long", "spare", "slot"):
        parents, table, idx, lens, spare, pools, dtype = reorder_case(rng, 2, 3, 16, 40)
        lens[:] = 0
        table[:] = -7
        lens[:3], lens[3:] = 21, 37
        ids = list(range(6, 6 + 2 * 3 + 3 * 3))
        total = 6 + 15
        spare[:] = range(6)
        for i in range(6):
            for c in range(-(-lens[i] // 16)):
                p = ids.pop()
                j = np.arange(c * 16, min(c * 16 + 16, lens[i]))
                table[idx[i], j] = p * 16 + j % 16
        pools = [torch.from_numpy(rng.integers(0, 256, (total, 16, 2, 128), dtype=np.uint8)) for _ in range(2)]
        parents[:] = [[1, 2, 0], [2, 0, 1]]
        bad = dict(parents=parents.copy(), idx=idx.copy(), lens=lens.copy(), spare=spare.copy(), table=table.copy())
        bits = pa.PA_DEVERR_TABLE_INDEX
        if what == "parent":
            bad["parents"][0, 1] = 3
        elif what == "negative_parent":
            bad["parents"][0, 1] = -1
        elif what == "idx":
            bad["idx"][1] = table.shape[0]
        elif what == "length":
            bad["lens"][1], bits = 22, pa.PA_DEVERR_SEQLENS
        elif what == "long":
            bad["lens"][:3], bits = 1000, pa.PA_DEVERR_SEQLENS
        elif what == "spare":
            bad["spare"][1], bits = total, pa.PA_DEVERR_PAGE_RANGE
        else:
            bad["table"][idx[2], 20], bits = -7, pa.PA_DEVERR_PAGE_RANGE
        d = lambda a: torch.from_numpy(np.array(a)).to(cuda_device)
        t, s = d(bad["table"]), d(bad["spare"])
        dp = [p.to(cuda_device).view(torch.bfloat16) for p in pools]
        pa.beam_reorder(d(bad["parents"]), t, d(bad["idx"]), d(bad["lens"]), s, dp[0], dp[1])
        assert pa.device_error() & bits, what
        want = [p.flatten(2).numpy().copy() for p in pools]
        plain_reorder(parents[1:], table, idx[3:], lens[3:], spare[3:], want, 16)
        assert np.array_equal(t.cpu().numpy()[idx[3:]], table[idx[3:]]), what
        assert np.array_equal(s.cpu().numpy()[3:], spare[3:]), what
        for p, w in zip(dp, want):
            assert np.array_equal(p.view(torch.uint8).flatten(2).cpu().numpy()[3:6], w[3:6]), what
