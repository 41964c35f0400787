"""Decode over shared prefixes against a 64-bit implementation.

Tolerances, from the arithmetic (A = the attention over |V|):
  - the output is rounded to bf16 once: 2^-8 |o|;
  - P is rounded to bf16 over bf16 pools (2^-8 of each weight, the sum of weights
    in 32 bits: 2^-8 A at most) or to f16 over the others (2^-11 A); FP8 pools
    round q * k_scale to f16 as well: each product q k is off by 2^-11 of itself,
    a score by 2^-11 sum|q k| scale, below 2^-11 * 40 for these inputs (the rest
    of a score's error, 128 * 2^-24 of the same sum, is below 2^-12);
  - lse: the scores' errors: 3e-4, and 2^-11 * 40 over FP8 pools.
"""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FP8 = 1
FP4 = 2


def make(dev, seed, sizes, prefixes, tails, hq, hkv, d, page, kv, loose=0):
    """A batch: len(sizes) groups and `loose` sequences of none; the slots that no
    key uses hold NaN.  tails: keys behind the prefix per sequence."""
    import paged_kv_flashattention_gb300 as pa
    rng = random.Random(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    first = [p for p, n in zip(prefixes, sizes) for _ in range(n)] + [0] * loose
    B = len(first)
    lens = [p + t for p, t in zip(first, tails)]
    cols = max(1, max([-(-n // page) for n in lens], default=1))
    need = sum(p // page for p in prefixes) + sum(-(-n // page) - f // page for n, f in zip(lens, first))
    ids = list(range(need + 2))
    rng.shuffle(ids)
    poison = ids.pop()
    table = np.full((B, cols), poison, np.int32)
    copies, b = [], 0
    for p, n in zip(prefixes, sizes):
        whole = [ids.pop() for _ in range(p // page)]
        for q in range(b, b + n):
            table[q, :len(whole)] = whole
            if p % page and q > b:
                copies.append((b, q, p))
        b += n
    for q in range(B):
        for c in range(first[q] // page, -(-lens[q] // page)):
            table[q, c] = ids.pop()
    slots = (need + 2) * page
    live = np.zeros(slots, bool)
    for q in range(B):
        j = np.arange(lens[q])
        live[table[q, j // page].astype(np.int64) * page + j % page] = True
    x = [torch.randn((slots, hkv, d), generator=g, device=dev).bfloat16() for _ in range(2)]
    for a, q, p in copies:
        j = np.arange(p // page * page, p)
        for v in x:
            v[torch.as_tensor(table[q, p // page] * page + j % page, device=dev)] = \
                v[torch.as_tensor(table[a, p // page] * page + j % page, device=dev)]
    scales = {}
    if kv == 0:
        pools = [v.clone() for v in x]
        vals = [v.double() for v in x]
    else:
        ks = 4.5 / (448 if kv == FP8 else 2688) * (0.8 + 0.4 * torch.rand((2, hkv), generator=g, device=dev))
        scales = {"k_scale": ks[0].contiguous(), "v_scale": ks[1].contiguous()}
        slot = torch.arange(slots, dtype=torch.int32, device=dev)
        if kv == FP8:
            pools = [torch.zeros((slots, hkv, d), dtype=torch.uint8, device=dev) for _ in range(2)]
            pa.store_kv_fp8(x[0], x[1], slot, pools[0], pools[1], ks[0].contiguous(), ks[1].contiguous())
            vals = [p.view(torch.float8_e4m3fn).double() * s.double()[:, None] for p, s in zip(pools, ks)]
        else:
            pools = [torch.zeros((slots, pa.fp4_row_bytes(hkv, d)), dtype=torch.uint8, device=dev) for _ in range(2)]
            pa.store_kv_fp4(x[0], x[1], slot, pools[0], pools[1], ks[0].contiguous(), ks[1].contiguous())
            from oracle import fp4
            vals = [torch.from_numpy(fp4.unpack(p.cpu().numpy(), hkv, d, s.cpu().numpy())).to(dev).double()
                    for p, s in zip(pools, ks)]
        scales["kv_dtype"] = kv
    dead = torch.from_numpy(~live).to(dev)
    for p in pools:
        p[dead] = float("nan") if kv == 0 else 255
    pools = [p.view((need + 2, page) + tuple(p.shape[1:])) for p in pools]
    dv = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    q = torch.randn((B, hq, d), generator=g, device=dev).bfloat16()
    return dict(q=q, pools=pools, vals=vals, table=torch.from_numpy(table).to(dev), lens=dv(lens), first=dv(first),
                cu=dv(np.cumsum([0] + list(sizes)).tolist()), scales=scales, host=(lens, table, page, hkv),
                bounds=dict(max_prefix=max(prefixes, default=0), max_suffix=max(tails, default=0), max_group=max(sizes, default=0)),
                max_k=max(lens + [1]))


def reference(s):
    """(out, lse, attention over |V|) in 64 bits, each sequence by its own row
    (a prefix's last page is the same in every row)."""
    lens, table, page, hkv = s["host"]
    B, hq, d = s["q"].shape
    outs = []
    for b in range(B):
        if lens[b] == 0:
            z = torch.zeros((hq, d), dtype=torch.float64, device=s["q"].device)
            outs.append((z, torch.full((hq,), float("-inf"), dtype=torch.float64, device=z.device), z))
            continue
        j = np.arange(lens[b])
        slot = torch.as_tensor(table[b, j // page].astype(np.int64) * page + j % page, device=s["q"].device)
        k, v = (x[slot].permute(1, 0, 2) for x in s["vals"])
        x = (s["q"][b].double().view(hkv, hq // hkv, d) @ k.transpose(1, 2)) * d ** -0.5
        w = torch.softmax(x, -1)
        outs.append(((w @ v).reshape(hq, d), torch.logsumexp(x, -1).reshape(hq), (w @ v.abs()).reshape(hq, d)))
    return [torch.stack(t) for t in zip(*outs)]


def run(s, **kw):
    import paged_kv_flashattention_gb300 as pa
    lse = torch.full(s["q"].shape[:2], 7.0, dtype=torch.float32, device=s["q"].device)
    out = torch.full_like(s["q"], 7.0)
    args = {**s["bounds"], **s["scales"], **kw}
    pa.decode_shared(s["q"], *s["pools"], s["table"], s["lens"], s["max_k"], s["cu"], s["first"], out=out, lse=lse, **args)
    assert pa.device_error() == 0
    return out, lse


def check(s, got, rows=None):
    kv = s["scales"].get("kv_dtype", 0)
    want, want_l, mag = s["ref"] if "ref" in s else reference(s)
    out, lse = got[0].double(), got[1].double()
    if rows is not None:
        want, want_l, mag, out, lse = (t[rows] for t in (want, want_l, mag, out, lse))
    tol = 2.0 ** -8 * want.abs() + {0: 2.0 ** -8 + 2.0 ** -11, FP8: 2.0 ** -11 * 42, FP4: 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -13}[kv] * mag
    over = (out - want).abs() - tol
    assert bool((over <= 0).all()), f"{int((~(over <= 0)).sum())} of {over.numel()} outputs off, worst {float(over.max()):.3g}"
    empty = torch.isneginf(want_l)
    assert torch.equal(torch.isneginf(lse), empty)
    assert not bool(out[empty].any())
    err = (lse - want_l)[~empty].abs()
    assert err.numel() == 0 or float(err.max()) <= (2.0 ** -11 * 40 if kv == FP8 else 3e-4)


SHAPES = [  # hq, hkv, d, page
    (32, 8, 128, 16), (32, 8, 64, 16), (8, 8, 128, 1), (12, 6, 64, 16), (8, 1, 128, 16), (16, 2, 64, 1), (2, 1, 128, 1),
    (64, 16, 128, 16),
]


@pytest.mark.parametrize("kv", [0, FP8, FP4])
@pytest.mark.parametrize("shape", SHAPES)
def test_groups(cuda_device, shape, kv):
    """Ragged groups, one of them empty, prefixes that end inside pages and
    tiles, sequences without keys of their own, and sequences of no group."""
    hq, hkv, d, page = shape
    sizes, prefixes = [5, 1, 0, 17, 2], [300, 129, 64, 1000, 128]
    rng = random.Random(3)
    tails = [rng.choice([0, 1, 16, 37, 200]) for _ in range(sum(sizes) + 3)]
    s = make(cuda_device, 11, sizes, prefixes, tails, hq, hkv, d, page, kv, loose=3)
    check(s, run(s))


@pytest.mark.parametrize("kv", [0, FP8, FP4])
@pytest.mark.parametrize("n", [31, 32, 33, 64, 65, 130])
def test_group_sizes(cuda_device, n, kv):
    """A group's rows around one, two and four tiles of 128 (4 rows a sequence)."""
    s = make(cuda_device, n, [n], [700], [b % 20 for b in range(n)], 8, 2, 128, 16, kv)
    check(s, run(s))


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 5000])
@pytest.mark.parametrize("page", [1, 16])
def test_prefix_lengths(cuda_device, prefix, page):
    s = make(cuda_device, prefix, [3, 4], [prefix, max(0, prefix - 7)], [1, 0, 5, 16, 0, 33, 2], 8, 2, 64, page, 0)
    check(s, run(s))


@pytest.mark.parametrize("kv", [0, FP8, FP4])
def test_many_groups(cuda_device, kv):
    """More groups than threads of a CTA; most hold one sequence."""
    rng = random.Random(5)
    sizes = [rng.choice([0, 1, 1, 1, 2, 3]) for _ in range(700)]
    prefixes = [rng.choice([0, 1, 40, 128, 200]) for _ in sizes]
    s = make(cuda_device, 7, sizes, prefixes, [rng.randrange(4) for _ in range(sum(sizes))], 4, 2, 64, 16, kv)
    check(s, run(s))


def test_bounds_may_be_loose(cuda_device):
    import paged_kv_flashattention_gb300 as pa
    s = make(cuda_device, 1, [6, 2], [333, 48], [3, 9, 1, 0, 4, 70, 8, 8], 16, 4, 128, 16, 0)
    s["ref"] = reference(s)
    check(s, run(s))
    check(s, run(s, max_prefix=None, max_suffix=None, max_group=None))
    # one workspace for the larger call serves the smaller one, full of NaN before each
    kw = dict(max_prefix=s["max_k"], max_suffix=s["max_k"], max_group=8)
    need = pa.decode_shared_workspace_size(s["q"].shape, s["pools"][0], s["max_k"], 2, **kw)
    ws = torch.full((need // 4 + 1,), float("nan"), device=cuda_device)
    check(s, run(s, workspace=ws, **kw))
    ws.fill_(float("nan"))
    check(s, run(s, workspace=ws))


@pytest.mark.parametrize("kv", [0, FP8, FP4])
@pytest.mark.parametrize("prefix,tails,loose", [
    (16, (3000, 2500, 3001, 1), False), (9000, (0, 1, 0, 0), True), (9000, (0, 0, 0, 0), True), (4000, (4000, 10, 4000, 7), False),
    (20000, (3, 16, 1, 40), True),
])
def test_prefix_beside_tails(cuda_device, prefix, tails, loose, kv):
    """Prefixes and tails of every proportion, so that few and all of the CTAs take
    part in the prefix, under tight bounds and loose ones."""
    s = make(cuda_device, prefix + len(tails), [3, 2], [prefix, prefix // 2], [*tails, 5], 16, 8, 64, 16, kv)
    check(s, run(s, **(dict(max_prefix=None, max_suffix=None) if loose else {})))


def test_padding_rows(cuda_device):
    """Rows of length 0 inside a group with a prefix and behind all groups."""
    s = make(cuda_device, 2, [4, 3], [200, 100], [3, 5, 0, 7, 1, 2, 3, 0], 8, 2, 128, 16, 0, loose=1)
    s["lens"][2] = 0
    s["lens"][6] = 0
    s["host"][0][2] = s["host"][0][6] = 0
    check(s, run(s))


def test_equals_decode(cuda_device):
    """The same batch through pa.decode, within both paths' roundings."""
    import paged_kv_flashattention_gb300 as pa
    s = make(cuda_device, 4, [8, 8], [512, 1024], [17] * 16, 32, 8, 128, 16, 0)
    out, lse = run(s)
    lse2 = torch.empty_like(lse)
    out2 = pa.decode(s["q"], *s["pools"], s["table"], s["lens"], s["max_k"], lse=lse2)
    _, _, mag = reference(s)
    assert bool(((out.double() - out2.double()).abs() <= 2.0 ** -8 * (out2.double().abs() * 2 + 2.25 * mag)).all())
    assert float((lse - lse2).abs().max()) <= 6e-4


def test_runs_are_equal_and_capture(cuda_device):
    """Two runs give the same bits; a captured call follows lengths and groups
    that change between replays."""
    a = make(cuda_device, 21, [4, 4], [300, 200], [5, 1, 9, 2, 7, 7, 7, 7], 16, 4, 128, 16, 0)
    b = make(cuda_device, 22, [3, 5], [150, 410], [1, 2, 3, 4, 5, 6, 7, 8], 16, 4, 128, 16, 0)
    bounds = dict(max_prefix=512, max_suffix=16, max_group=8)
    one, two = run(a), run(a)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    import paged_kv_flashattention_gb300 as pa
    pages = max(a["pools"][0].shape[0], b["pools"][0].shape[0])
    fixed = {n: torch.zeros_like(a[n]) for n in ("q", "lens", "first", "cu")}
    table = torch.zeros((8, 40), dtype=torch.int32, device=cuda_device)
    pools = [torch.zeros((pages,) + tuple(p.shape[1:]), dtype=p.dtype, device=cuda_device) for p in a["pools"]]
    out, lse = torch.empty_like(a["q"]), torch.empty(a["q"].shape[:2], device=cuda_device)
    ws = torch.empty(pa.decode_shared_workspace_size(a["q"].shape, pools[0], 640, 2, **bounds), dtype=torch.uint8, device=cuda_device)

    def call():
        pa.decode_shared(fixed["q"], *pools, table, fixed["lens"], 640, fixed["cu"], fixed["first"], out=out, lse=lse,
                         workspace=ws, **bounds)

    def load(s):
        for n, t in fixed.items():
            t.copy_(s[n])
        table[:, :s["table"].shape[1]] = s["table"]
        for p, x in zip(pools, s["pools"]):
            p[:x.shape[0]] = x

    load(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    for s in (a, b, a):
        load(s)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert pa.device_error() == 0
        check(s, (out, lse))


def test_no_groups_is_decode(cuda_device):
    import paged_kv_flashattention_gb300 as pa
    s = make(cuda_device, 6, [], [], [100, 0, 33], 8, 2, 64, 16, 0, loose=3)
    out, lse = run(s)
    assert torch.equal(out, pa.decode(s["q"], *s["pools"], s["table"], s["lens"], s["max_k"]))
    check(s, (out, lse))


def test_wide_scores(cuda_device):
    """Scores of hundreds (the maximum moves from tile to tile)."""
    s = make(cuda_device, 9, [9], [900], [30] * 9, 8, 2, 128, 16, 0)
    s["q"].mul_(64)
    want, want_l, mag = reference(s)
    out, lse = run(s)
    # a score's error, 128 * 2^-24 * sum|q k| scale < 128 * 2^-24 * 64 * 11, is relative in p
    tol = 2.0 ** -8 * (want.abs() + mag) + 6e-3 * mag
    assert bool(((out.double() - want).abs() <= tol).all())
    assert float((lse.double() - want_l).abs().max()) <= 6e-3


@pytest.mark.parametrize("what", ["prefix_over_bound", "prefix_over_length", "differs", "no_group", "group_over_bound",
                                  "groups_backwards", "suffix_over_bound", "page"])
@pytest.mark.parametrize("kv", [0, FP4])
def test_bad_device_data(cuda_device, what, kv):
    """Data outside the call's bounds raises the error word; sequences that it
    does not concern keep their results."""
    import paged_kv_flashattention_gb300 as pa
    s = make(cuda_device, 8, [3, 3], [200, 96], [5, 6, 7, 8, 9, 10, 11, 12], 8, 2, 64, 16, kv, loose=2)
    s["ref"] = reference(s)
    bounds, good, bits = dict(s["bounds"]), None, pa.PA_DEVERR_SEQLENS
    if what == "prefix_over_bound":
        bounds["max_prefix"], good = 100, [3, 4, 5, 6, 7]
    elif what == "prefix_over_length":
        s["lens"][1], good = 150, [0, 2, 3, 4, 5, 6, 7]
    elif what == "differs":
        s["first"][1], good = 180, [0, 2, 3, 4, 5, 6, 7]
    elif what == "no_group":
        s["first"][7], good = 10, [0, 1, 2, 3, 4, 5, 6]
    elif what == "group_over_bound":
        bounds["max_group"], good = 2, [6, 7]
    elif what == "groups_backwards":
        s["cu"][1], good = 9, [6, 7]
    elif what == "suffix_over_bound":
        bounds["max_suffix"], good = 11, [0, 1, 2, 3, 4, 5, 6]
    else:
        s["table"][3, 2], good, bits = 1 << 30, [0, 1, 2, 6, 7], pa.PA_DEVERR_PAGE_RANGE
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=cuda_device)
    out = pa.decode_shared(s["q"], *s["pools"], s["table"], s["lens"], s["max_k"], s["cu"], s["first"], lse=lse, **bounds,
                           **s["scales"])
    assert pa.device_error() & bits
    check(s, (out, lse), rows=good)


def test_other_stream_and_two_calls(cuda_device):
    """Calls on two streams, a workspace each."""
    import paged_kv_flashattention_gb300 as pa
    batches = [make(cuda_device, 30 + i, [5, 9], [400, 900], [i + b for b in range(14)], 16, 4, 128, 16, 0) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = []
        for s, st in zip(batches, streams):
            with torch.cuda.stream(st):
                lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=cuda_device)
                out = pa.decode_shared(s["q"], *s["pools"], s["table"], s["lens"], s["max_k"], s["cu"], s["first"], lse=lse,
                                       **s["bounds"])
                outs.append((out, lse))
    torch.cuda.synchronize()
    for s, got in zip(batches, outs):
        check(s, got)
